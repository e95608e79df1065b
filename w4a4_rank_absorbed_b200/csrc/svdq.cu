// C ABI of the SVDQuant W4A4 linear layer (declared in include/svdq.h):
// argument checks, TMA descriptor encoding and kernel launches.
// All kernels live in this one translation unit so they share one device
// error word.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <utility>

#include "../../include/svdq.h"
#include "common.cuh"
#include "calib.cuh"
#include "group_norm.cuh"
#include "linear.cuh"
#include "linear_i8.cuh"
#include "pack_weight.cuh"
#include "quantize_act.cuh"

namespace {

using namespace svdq;

constexpr int kMaxDevices = 64;

// ----------------------------------------------------------- device info ----
struct DevInfo {
  bool init = false;
  bool ok = false;
  int sms = 0;
  bool linear_attr[3] = {};     // [NVFP4, MXFP4, NVFP4 with the GELU + next-layer quantization epilogue]
  bool qa_attr[3][9] = {};      // [NVFP4 quantize, down-projection only, MXFP4 quantize][r / 16]
};
DevInfo g_dev[kMaxDevices];
std::mutex g_mu;

svdq_status current_device(int* dev_out, DevInfo** info) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SVDQ_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return SVDQ_ERR_DEVICE;
  std::lock_guard<std::mutex> lk(g_mu);
  DevInfo& d = g_dev[dev];
  if (!d.init) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return SVDQ_ERR_CUDA;
    d.ok = (major == 10 && minor == 0);
    d.sms = sms;
    d.init = true;
  }
  if (!d.ok) return SVDQ_ERR_DEVICE;
  *dev_out = dev;
  *info = &d;
  return SVDQ_OK;
}

// ------------------------------------------------------------ TMA maps ------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 2-D row-major tensor (rows x inner elements, row pitch in bytes), box (box_inner x box_rows),
// 128-byte swizzle unless stated.
// Tensor maps are cached on the host: a call on the same buffers with the same shapes (every forward
// pass of a layer) reuses the encoded map instead of encoding it again.  A map holds only the
// address, the shape and the box, so a cached entry stays valid for any later buffer at the same
// address with the same shape.  64 entries, least recently used replaced, one mutex.
struct MapKey {
  const void* base;
  uint32_t dt, rank, swizzle;
  uint64_t dims[3], strides[2];
  uint32_t box[3];
  bool operator==(const MapKey& o) const {
    return base == o.base && dt == o.dt && rank == o.rank && swizzle == o.swizzle &&
           std::memcmp(dims, o.dims, sizeof(dims)) == 0 && std::memcmp(strides, o.strides, sizeof(strides)) == 0 &&
           std::memcmp(box, o.box, sizeof(box)) == 0;
  }
};
struct MapEntry {
  MapKey key;
  CUtensorMap map;
  uint64_t stamp = 0;
  bool used = false;
};
constexpr int kMapCacheEntries = 64;
MapEntry g_maps[kMapCacheEntries];
uint64_t g_map_clock = 0;
uint64_t g_map_hits = 0, g_map_misses = 0;
std::mutex g_map_mu;

bool encode_map(const MapKey& k, CUtensorMap* m) {
  {
    std::lock_guard<std::mutex> lk(g_map_mu);
    for (MapEntry& e : g_maps)
      if (e.used && e.key == k) {
        e.stamp = ++g_map_clock;
        *m = e.map;
        ++g_map_hits;
        return true;
      }
  }
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {k.dims[0], k.dims[1], k.dims[2]};
  cuuint64_t strides[2] = {k.strides[0], k.strides[1]};
  cuuint32_t box[3] = {k.box[0], k.box[1], k.box[2]};
  cuuint32_t estr[3] = {1, 1, 1};
  if (fn(m, (CUtensorMapDataType)k.dt, k.rank, const_cast<void*>(k.base), dims, strides, box, estr,
         CU_TENSOR_MAP_INTERLEAVE_NONE, (CUtensorMapSwizzle)k.swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  std::lock_guard<std::mutex> lk(g_map_mu);
  MapEntry* victim = &g_maps[0];
  for (MapEntry& e : g_maps) {
    if (!e.used) {
      victim = &e;
      break;
    }
    if (e.stamp < victim->stamp) victim = &e;
  }
  victim->key = k;
  victim->map = *m;
  victim->stamp = ++g_map_clock;
  victim->used = true;
  ++g_map_misses;
  return true;
}

bool make_map_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t rows,
                 uint64_t pitch_bytes, uint32_t box_inner, uint32_t box_rows,
                 CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  MapKey k{};
  k.base = base;
  k.dt = (uint32_t)dt;
  k.rank = 2;
  k.swizzle = (uint32_t)swizzle;
  k.dims[0] = inner;
  k.dims[1] = rows;
  k.strides[0] = pitch_bytes;
  k.box[0] = box_inner;
  k.box[1] = box_rows;
  return encode_map(k, m);
}

// The rows x K bf16 matrix at `base` as a 3-D tensor {64 columns, rows, K/64 chunks} (strides 2K and
// 128 bytes), box {64, box_rows, 2}, 128-byte swizzle: one copy brings two adjacent 64-column
// chunks of box_rows rows and lands them as two 128-byte-swizzled tiles, one after the other.
bool make_map_chunks(CUtensorMap* m, const void* base, uint64_t K, uint64_t rows, uint32_t box_rows) {
  MapKey k{};
  k.base = base;
  k.dt = (uint32_t)CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  k.rank = 3;
  k.swizzle = (uint32_t)CU_TENSOR_MAP_SWIZZLE_128B;
  k.dims[0] = 64;
  k.dims[1] = rows;
  k.dims[2] = K / 64;
  k.strides[0] = K * 2;
  k.strides[1] = 128;
  k.box[0] = 64;
  k.box[1] = box_rows;
  k.box[2] = 2;
  return encode_map(k, m);
}

// ------------------------------------------------------------- checks -------
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

// M = 0 (an empty batch) passes; the per-forward entry points then return SVDQ_OK at once.
svdq_status check_shape(int64_t M, int64_t N, int64_t K, int r) {
  if (M < 0 || N < 1 || K < 1 || r < 0) return SVDQ_ERR_INVALID_ARG;
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (K % 64 != 0 || N % 16 != 0 || r % 16 != 0 || r > 128) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  return SVDQ_OK;
}

svdq_status launch_status() {
  return cudaGetLastError() == cudaSuccess ? SVDQ_OK : SVDQ_ERR_CUDA;
}

int64_t pad128(int64_t v) { return (v + 127) / 128 * 128; }

// Launch as a programmatic dependent of the previous kernel on the stream: the kernel's prologue
// (barrier set-up, TMEM allocation, descriptor prefetch) overlaps that kernel's tail, and the kernel
// waits for it (griddepcontrol.wait) before it touches global memory.  cluster > 1 launches
// thread-block clusters of that many CTAs along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, int cluster,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  int n = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    n = 2;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// --------------------------------------------------------- quantize_act -----
// CTAs that share a 128-row block split its K chunks between them: the smallest split in
// {1, 2, 4, 8} that gives about one CTA per SM (the kernel runs one 576-thread CTA per SM, so a
// larger grid would run in two waves), with at least two chunks a CTA.
int qa_split(int64_t M, int64_t K, int sms) {
  const int64_t rb = pad128(M) / 128, nunits = (K / 64 + 1) / 2;   // stages of two 64-column chunks
  int split = 1;
  while (split < QB_MAX_SPLIT && rb * 2 * split <= (int64_t)sms && nunits >= 2 * split) split *= 2;
  return split;
}

// Workspace of kernel 2 (see include/svdq.h): the ticket words first, then the partial sums.
size_t qa_ticket_bytes(int64_t M) { return (size_t)((pad128(M) / 128 * 4 + 255) / 256 * 256); }
size_t qa_workspace_bytes(int64_t M, int r) {
  return r > 0 ? qa_ticket_bytes(M) + (size_t)QB_MAX_SPLIT * (size_t)pad128(M) * (size_t)r * 4 : 0;
}

// ------------------------------------------------ scratch of svdq_quantize_act_noalloc ---
// Device memory the library owns for callers that cannot allocate: the counters and partial sums
// of kernel 2's K split.  In host code the name stands for a host-side handle, not a device address,
// so the kernels are given the address cudaGetSymbolAddress returns for the current device.
constexpr size_t kNoAllocScratchBytes = SVDQ_NOALLOC_SCRATCH_BYTES;
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];
void* g_noalloc_ptr[kMaxDevices] = {};

// Bytes of the scratch a call uses: the counters, then the partial sums of the split the launch takes.
size_t noalloc_scratch_need(int64_t M, int64_t K, int r, int sms) {
  return qa_ticket_bytes(M) + (size_t)qa_split(M, K, sms) * (size_t)pad128(M) * (size_t)r * 4;
}

// Device address of the scratch array on device `dev` (the current device), looked up once.
svdq_status noalloc_scratch(int dev, DevInfo* d, void** out) {
  (void)d;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_noalloc_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || !p) return SVDQ_ERR_CUDA;
    g_noalloc_ptr[dev] = p;
  }
  *out = g_noalloc_ptr[dev];
  return SVDQ_OK;
}

template <int R, bool QUANT, bool MX = false>
svdq_status launch_qa(DevInfo* d, const uint16_t* X, int64_t M, int64_t K, const float* inv_s, float gs_x,
                      const uint16_t* L1fT, float lr_scale, uint8_t* Xq, uint8_t* SFx, uint16_t* LAs,
                      void* ws, cudaStream_t s) {
  using Cfg = QbCfg<R>;
  CUtensorMap tm_x, tm_l1, tm_x1, tm_l11;
  if (!make_map_chunks(&tm_x, X, (uint64_t)K, (uint64_t)M, QB_ROWS) ||
      !make_map_2d(&tm_x1, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, X, (uint64_t)K, (uint64_t)M, (uint64_t)K * 2, 64,
                   QB_ROWS))
    return SVDQ_ERR_CUDA;
  if (R > 0) {
    if (!make_map_chunks(&tm_l1, L1fT, (uint64_t)K, (uint64_t)R, R > 0 ? R : 1) ||
        !make_map_2d(&tm_l11, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, L1fT, (uint64_t)K, (uint64_t)R, (uint64_t)K * 2, 64,
                     R > 0 ? R : 1))
      return SVDQ_ERR_CUDA;
  } else {
    tm_l1 = tm_x;
    tm_l11 = tm_x1;
  }
  bool& attr = d->qa_attr[MX ? 2 : QUANT ? 0 : 1][R / 16];
  if (!attr) {
    if (cudaFuncSetAttribute(k_quantize_act<R, QUANT, MX>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg::kSmem) != cudaSuccess)
      return SVDQ_ERR_CUDA;
    attr = true;
  }
  const int64_t Mpad = pad128(M);
  const int split = qa_split(M, K, d->sms);   // with r = 0 the CTAs of a row block only share out K
  unsigned int* ticket = reinterpret_cast<unsigned int*>(ws);
  float* part = ws ? reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + qa_ticket_bytes(M)) : nullptr;
  if (R > 0 && split > 1 && !ws) return SVDQ_ERR_INVALID_ARG;
  const dim3 grid((unsigned)(Mpad / QB_ROWS * split));
  if (launch_pdl(k_quantize_act<R, QUANT, MX>, grid, dim3(QB_THREADS), (size_t)Cfg::kSmem, s, 1, tm_x, tm_l1, tm_x1,
                 tm_l11, inv_s, gs_x, lr_scale, (int)M, (int)K, (int)Mpad, split, Xq, SFx, LAs, part, ticket,
                 LN_DEFAULT_TIMEOUT_NS) != cudaSuccess)
    return SVDQ_ERR_CUDA;
  return launch_status();
}

template <bool QUANT, bool MX = false>
svdq_status dispatch_qa(DevInfo* d, int r, const uint16_t* X, int64_t M, int64_t K, const float* inv_s, float gs_x,
                        const uint16_t* L1fT, float lr_scale, uint8_t* Xq, uint8_t* SFx, uint16_t* LAs,
                        void* ws, cudaStream_t s) {
  switch (r) {
    case 0:
      if (QUANT) return launch_qa<0, true, MX>(d, X, M, K, inv_s, gs_x, L1fT, lr_scale, Xq, SFx, LAs, ws, s);
      return SVDQ_ERR_INVALID_ARG;
    case 16: return launch_qa<16, QUANT, MX>(d, X, M, K, inv_s, gs_x, L1fT, lr_scale, Xq, SFx, LAs, ws, s);
    case 32: return launch_qa<32, QUANT, MX>(d, X, M, K, inv_s, gs_x, L1fT, lr_scale, Xq, SFx, LAs, ws, s);
    case 48: return launch_qa<48, QUANT, MX>(d, X, M, K, inv_s, gs_x, L1fT, lr_scale, Xq, SFx, LAs, ws, s);
    case 64: return launch_qa<64, QUANT, MX>(d, X, M, K, inv_s, gs_x, L1fT, lr_scale, Xq, SFx, LAs, ws, s);
    case 80: return launch_qa<80, QUANT, MX>(d, X, M, K, inv_s, gs_x, L1fT, lr_scale, Xq, SFx, LAs, ws, s);
    case 96: return launch_qa<96, QUANT, MX>(d, X, M, K, inv_s, gs_x, L1fT, lr_scale, Xq, SFx, LAs, ws, s);
    case 112: return launch_qa<112, QUANT, MX>(d, X, M, K, inv_s, gs_x, L1fT, lr_scale, Xq, SFx, LAs, ws, s);
    case 128: return launch_qa<128, QUANT, MX>(d, X, M, K, inv_s, gs_x, L1fT, lr_scale, Xq, SFx, LAs, ws, s);
    default: return SVDQ_ERR_UNSUPPORTED_SHAPE;
  }
}

// The next layer's quantization done in the GEMM epilogue (svdq_linear_gelu_quantize).
struct GqArgs {
  const float* inv_s2;
  float gs_x2;
  const uint16_t* L1fT2;
  int r2;
  float lr_scale2;
  uint8_t* Xq2;
  uint8_t* SFx2;
  uint16_t* LAs2;
  float* part;
};

size_t gq_workspace_bytes(int64_t M, int64_t N, int r2) {
  if (r2 <= 0) return 0;
  return (size_t)((N + LN_BN - 1) / LN_BN) * (size_t)pad128(M) * (size_t)r2 * sizeof(float);
}

svdq_status linear_impl(const uint8_t* Xq, const uint8_t* SFx, float gs_x, const uint8_t* Wq, const uint8_t* SFw,
                        float gs_w, const uint16_t* LAs, const uint16_t* L2p, int r, const uint16_t* bias, void* Y,
                        int y_fp32, int64_t M, int64_t N, int64_t K, int debug, uint64_t timeout_ns,
                        cudaStream_t s, int y_accum = 0, bool mx = false, const GqArgs* gq = nullptr) {
  // y_accum: the rank-only mode (no 4-bit operands, K = 0) that adds the up-projection into Y.
  // gq: no Y; the epilogue writes the next layer's quantized activations instead.
  svdq_status st = check_shape(M, N, y_accum ? 64 : K, r);
  if (st != SVDQ_OK) return st;
  if (mx && K % 128 != 0) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return (y_accum && r == 0) ? SVDQ_ERR_INVALID_ARG : SVDQ_OK;   // an empty batch: nothing to launch
  if (y_accum ? (r == 0 || !LAs || !L2p || !Y || bias)
              : (!Xq || !SFx || !Wq || !SFw || (!gq && !Y) || (r > 0 && (!LAs || !L2p))))
    return SVDQ_ERR_INVALID_ARG;
  if (y_fp32 != 0 && y_fp32 != 1) return SVDQ_ERR_INVALID_ARG;
  if ((!y_accum && (!aligned16(Xq) || !aligned16(SFx) || !aligned16(Wq) || !aligned16(SFw))) ||
      (!gq && !aligned16(Y)) || (bias && !aligned16(bias)) || (r > 0 && (!aligned16(LAs) || !aligned16(L2p))))
    return SVDQ_ERR_MISALIGNED;
  if (gq) {
    if (N % 64 != 0 || (gq->r2 != 0 && gq->r2 != 16 && gq->r2 != 32)) return SVDQ_ERR_UNSUPPORTED_SHAPE;
    if (!gq->inv_s2 || !gq->Xq2 || !gq->SFx2 || !(gq->gs_x2 > 0.0f) || !std::isfinite(gq->gs_x2) ||
        (gq->r2 > 0 && (!gq->L1fT2 || !gq->LAs2 || !gq->part)))
      return SVDQ_ERR_INVALID_ARG;
    if (!aligned16(gq->inv_s2) || !aligned16(gq->Xq2) || !aligned16(gq->SFx2) ||
        (gq->r2 > 0 && (!aligned16(gq->L1fT2) || !aligned16(gq->LAs2) || !aligned16(gq->part))))
      return SVDQ_ERR_MISALIGNED;
  }
  int dev;
  DevInfo* d;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;

  CUtensorMap tm_xq, tm_wq, tm_las, tm_l2p;
  if (!y_accum &&
      (!make_map_2d(&tm_xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, Xq, (uint64_t)K / 2, (uint64_t)M, (uint64_t)K / 2, 128,
                    LN_BM) ||
       !make_map_2d(&tm_wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, Wq, (uint64_t)K / 2, (uint64_t)N, (uint64_t)K / 2, 128,
                    LN_BN / 2)))
    return SVDQ_ERR_CUDA;
  if (r > 0) {
    if (!make_map_2d(&tm_las, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, LAs, (uint64_t)2 * r, (uint64_t)M,
                     (uint64_t)4 * r, 64, LN_BM) ||
        !make_map_2d(&tm_l2p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, L2p, (uint64_t)r, (uint64_t)N,
                     (uint64_t)2 * r, 32, LN_BN / 2, CU_TENSOR_MAP_SWIZZLE_64B))
      return SVDQ_ERR_CUDA;
  } else {
    tm_las = tm_xq;
    tm_l2p = tm_wq;
  }
  if (y_accum) {                 // no K tiles: the 4-bit maps are never used
    tm_xq = tm_las;
    tm_wq = tm_l2p;
  }
  const int variant = gq ? 2 : mx ? 1 : 0;
  auto kernel = gq ? k_linear<false, true> : mx ? k_linear<true, false> : k_linear<false, false>;
  const int smem_bytes = gq ? LN_SMEM_GQ : LN_SMEM;
  if (!d->linear_attr[variant]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes) != cudaSuccess)
      return SVDQ_ERR_CUDA;
    d->linear_attr[variant] = true;
  }
  LinearArgs a;
  a.SFx = SFx;
  a.SFw = SFw;
  a.bias = bias;
  a.Y = Y;
  a.y_fp32 = y_fp32;
  a.y_vec32 = (reinterpret_cast<uintptr_t>(Y) & 31u) == 0 ? 1 : 0;
  a.y_accum = y_accum;
  a.M = (int)M;
  a.N = (int)N;
  a.K = y_accum ? 0 : (int)K;
  a.r = r;
  a.gs = gs_x * gs_w;
  a.debug = debug;
  a.timeout_ns = timeout_ns ? timeout_ns : LN_DEFAULT_TIMEOUT_NS;
  a.inv_s2 = gq ? gq->inv_s2 : nullptr;
  a.gs_x2 = gq ? gq->gs_x2 : 1.0f;
  a.L1fT2 = gq ? gq->L1fT2 : nullptr;
  a.r2 = gq ? gq->r2 : 0;
  a.Mpad = (int)pad128(M);
  a.Xq2 = gq ? gq->Xq2 : nullptr;
  a.SFx2 = gq ? gq->SFx2 : nullptr;
  a.part = gq ? gq->part : nullptr;
  const int64_t tiles = ((M + LN_BM - 1) / LN_BM) * ((N + LN_BN - 1) / LN_BN);
  const int grid = (int)(tiles < d->sms ? tiles : d->sms);
  if (launch_pdl(kernel, dim3(grid), dim3(LN_THREADS), (size_t)smem_bytes, s, 1, tm_xq, tm_wq, tm_las, tm_l2p, a) !=
      cudaSuccess)
    return SVDQ_ERR_CUDA;
  if (gq && gq->r2 > 0) {
    const int items = (int)M * (gq->r2 / 4);
    if (launch_pdl(k_lowrank_finalize, dim3((items + 255) / 256), dim3(256), 0, s, 1, (const float*)gq->part,
                   (int)((N + LN_BN - 1) / LN_BN), (int)M, (int)pad128(M), gq->r2, gq->lr_scale2, gq->LAs2) !=
        cudaSuccess)
      return SVDQ_ERR_CUDA;
  }
  return launch_status();
}

// ------------------------------------------------------------- int8 layer ---
constexpr int64_t kMaxK8 = int64_t(1) << 17;      // 128 * 128 * K stays inside the 32-bit sum below this
constexpr int64_t kMaxRows8 = (int64_t(1) << 31) - 1024;   // rows and columns, rounded up to tiles, stay in 32 bits

// A call that failed to launch: its error must not be taken for a later call's.
svdq_status launch_failed() {
  (void)cudaGetLastError();
  return SVDQ_ERR_CUDA;
}

size_t dtype_size(int type) { return type == SVDQ_FP32 ? 4 : 2; }
bool dtype_ok(int type) { return type == SVDQ_BF16 || type == SVDQ_FP32 || type == SVDQ_FP16; }

svdq_status check_shape_i8(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 1 || K < 1) return SVDQ_ERR_INVALID_ARG;
  if (M > kMaxRows8 || N > kMaxRows8 || K >= kMaxK8 || K % 16 != 0) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  return SVDQ_OK;
}

// Rows of `width` elements at pitch ld, at `p`: NULL, pitch and alignment (row_align: every row on 16 bytes).
svdq_status check_rows(const void* p, int type, int64_t width, int64_t ld, bool row_align) {
  if (!p || ld < width) return SVDQ_ERR_INVALID_ARG;
  if (ld > (int64_t(1) << 37)) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(p) || (row_align && ((uint64_t)ld * dtype_size(type)) % 16 != 0)) return SVDQ_ERR_MISALIGNED;
  return SVDQ_OK;
}

template <typename T, int VPT, bool WARP>
cudaError_t run_quantize_i8(DevInfo* d, const T* X, int64_t M, int64_t K, int64_t ldx, const float* inv_s, int8_t* Xq,
                            float* sx, cudaStream_t s) {
  const int threads = WARP ? 256 : (int)((K / 8 + VPT - 1) / VPT + 31) / 32 * 32;
  const int rows = WARP ? 8 : 1;                                     // rows a block takes at a time
  // As many blocks as are at work at one time: each then fetches rows ahead of the ones it reduces.
  static std::atomic<int> resident[QI_MAX_THREADS / 32 + 1];         // per SM, by warps of a block; 0: not asked yet
  int per_sm = resident[threads / 32].load(std::memory_order_relaxed);
  if (per_sm == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k_quantize_act_i8<T, VPT, WARP>, threads, 0) !=
        cudaSuccess)
      return cudaErrorUnknown;
    resident[threads / 32].store(per_sm = std::max(1, per_sm), std::memory_order_relaxed);
  }
  const int64_t blocks = std::min<int64_t>((M + rows - 1) / rows, (int64_t)d->sms * per_sm);
  return launch_pdl(k_quantize_act_i8<T, VPT, WARP>, dim3((unsigned)blocks), dim3(threads), 0, s, 1, X, M, (int)K, ldx,
                    inv_s, Xq, sx);
}
template <typename T>
svdq_status quantize_i8(DevInfo* d, const void* Xv, int64_t ldx, int64_t M, int64_t K, const float* inv_s, int8_t* Xq,
                        float* sx, cudaStream_t s) {
  const T* X = static_cast<const T*>(Xv);
  const int64_t nv = K / 8;                                          // vectors of 8 in a row
  const bool warps = M > 4 * (int64_t)d->sms;                        // enough rows for a warp each
  const cudaError_t e =
      warps && nv <= 32    ? run_quantize_i8<T, 1, true>(d, X, M, K, ldx, inv_s, Xq, sx, s)
      : warps && nv <= 64  ? run_quantize_i8<T, 2, true>(d, X, M, K, ldx, inv_s, Xq, sx, s)
      : warps && nv <= 128 ? run_quantize_i8<T, 4, true>(d, X, M, K, ldx, inv_s, Xq, sx, s)
      : nv <= 1024         ? run_quantize_i8<T, 2, false>(d, X, M, K, ldx, inv_s, Xq, sx, s)
      : nv <= 2048         ? run_quantize_i8<T, 4, false>(d, X, M, K, ldx, inv_s, Xq, sx, s)
                           : launch_pdl(k_quantize_long_i8<T>, dim3((unsigned)M), dim3(QI_MAX_THREADS), 0, s, 1, X,
                                        (int)K, ldx, inv_s, Xq, sx);
  return e == cudaSuccess ? launch_status() : launch_failed();
}
svdq_status launch_quantize_i8(DevInfo* d, const void* X, int x_type, int64_t ldx, int64_t M, int64_t K,
                               const float* inv_s, int8_t* Xq, float* sx, cudaStream_t s) {
  if (x_type == SVDQ_BF16) return quantize_i8<__nv_bfloat16>(d, X, ldx, M, K, inv_s, Xq, sx, s);
  if (x_type == SVDQ_FP16) return quantize_i8<__half>(d, X, ldx, M, K, inv_s, Xq, sx, s);
  return quantize_i8<float>(d, X, ldx, M, K, inv_s, Xq, sx, s);
}

// Shared memory a kernel may use, raised once per device and kernel.
template <typename F>
svdq_status allow_smem(F kernel, int dev, std::atomic<bool> (&done)[kMaxDevices], int bytes) {
  if (done[dev].load(std::memory_order_acquire)) return SVDQ_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return launch_failed();
  done[dev].store(true, std::memory_order_release);
  return SVDQ_OK;
}

int y_vector(const void* Y, int type, int64_t ldy) {
  const uint64_t pitch = (uint64_t)ldy * dtype_size(type);
  if (pitch % 16 != 0) return 0;
  return pitch % 32 == 0 && (reinterpret_cast<uintptr_t>(Y) & 31u) == 0 ? 2 : 1;
}

std::atomic<bool> g_pair_attr[kMaxDevices], g_split_attr[kMaxDevices];

// Which kernel, tile and K split serve a shape: the least of the times (microseconds) these lines predict,
// fitted to a sweep of M 16..16384 by (N, K) of 320..12288 on a B200; a stage is 128 of K.
//   pair kernel, nt channels a tile:   2.6 + main + (waves - 1) max(main, 1.65 + 0.0068 nt) + 0.3 + 0.0095 nt,
//                                      main = stages (0.11 + 0.001 nt); later tiles hide their epilogue or wait for it
//   split kernel, nt tokens, split s:  2.9 + 0.7 (s > 1: cluster reduction)
//                                      + waves ((stages / s) (0.085 + 0.0015 nt) + nt (0.008 + 0.022 / s))
// Splits of 5 and 7 are left out: clusters of that size leave SMs of a GPC idle.
// (measured, both sides: 512 x 320 of K = 320: split nt 16 3.5 us, pair nt 64 4.1; 128 x 4096 of K = 4096: split
// nt 64, s 2 7.9, pair nt 64 9.0; 256 x 4096 of K = 4096: pair nt 64 8.9, split nt 64, s 2 10.7.)
// strips: in how many strips of columns the tiles of the pair kernel's last round are taken, where they are few: main and
// the last terms are then those of nt / strips, and 1 more (measured: 16384 x 1280 of K = 1280 26.5 us with two strips,
// 28.4 with whole tiles of the best width; 4096 x 4096 of K = 4096 46.5 and 48.1; 5120 x 4000 of K = 2048, where whole
// tiles are foreseen 0.4 slower, 32.1 and 31.4).
struct LinearI8Plan {
  bool pair;
  int nt, split, strips;
};
LinearI8Plan find_plan_linear_i8(int64_t M, int64_t N, int64_t K, int sms) {
  const int64_t nkt = (K + 127) / 128;
  LinearI8Plan best = {true, 256, 1, 1};
  double least = 1e30;
  const auto waves = [](int64_t tiles, int64_t at_once) { return (double)((tiles + at_once - 1) / at_once); };
  for (int nt = 256; nt >= 64; nt -= 32) {
    const int64_t tiles = (M + 255) / 256 * ((N + nt - 1) / nt);
    const double main = (double)nkt * (0.11 + 0.001 * nt), rest = 1.65 + 0.0068 * nt, w = waves(tiles, sms / 2);
    for (const int q : {1, 2, 4}) {
      const int64_t few = tiles % (sms / 2);
      if (q > 1 && (tiles < sms / 2 || few == 0 || few * q > sms / 2 || nt % (32 * q) != 0 || nt / q < 64)) continue;
      const double last = (double)nkt * (0.11 + 0.001 * (nt / q));
      const double t = 2.6 + (w - 1) * std::max(main, rest) + (q == 1 ? main : std::max(last, rest) + 1.0) + 0.3 +
                       0.0095 * (nt / q);
      if (t < least) {
        least = t;
        best = {true, nt, 1, q};
      }
    }
  }
  const int m16 = (int)std::min<int64_t>((M + 15) / 16 * 16, 128);   // all the tokens, where they fit a tile
  for (int nt = 16; nt <= 128; nt *= 2) {
    const int tok = std::min(nt, m16);
    const int64_t tiles = (M + tok - 1) / tok * ((N + 127) / 128);
    if (tiles > 4 * (int64_t)sms || (M + tok - 1) / tok > 65535) continue;
    for (const int s : {1, 2, 3, 4, 6, 8}) {
      if (s > 1 && (tiles * s > sms || 2 * s > nkt)) break;
      const double t = 2.9 + (s > 1 ? 0.7 : 0.0) +
                       waves(tiles * s, sms) * ((double)((nkt + s - 1) / s) * (0.085 + 0.0015 * tok) +
                                                tok * (0.008 + 0.022 / s));
      if (t < least) {
        least = t;
        best = {false, tok, s, 1};
      }
    }
    if (nt >= m16) break;
  }
  return best;
}

// The last plan of each calling thread is kept: a layer's calls are alike, and the search costs half a microsecond.
LinearI8Plan plan_linear_i8(int64_t M, int64_t N, int64_t K, int sms) {
  static thread_local struct {
    int64_t M = 0, N = 0, K = 0;
    int sms = 0;
    LinearI8Plan plan;
  } last;
  if (last.M != M || last.N != N || last.K != K || last.sms != sms) {
    last.plan = find_plan_linear_i8(M, N, K, sms);
    last.M = M;
    last.N = N;
    last.K = K;
    last.sms = sms;
  }
  return last.plan;
}

// Whether svdq_forward_i8 leaves the quantizing to the split kernel: where a half warp a chunk of 128 columns is enough.
// Measured, one launch against two, weights from HBM: 1 x 12288 of K = 4096 11.9 and 13.7 us, 1 x 4096 of K = 4096
// 6.7 and 8.5, 1 x 5120 of K = 1280 4.7 and 5.6, 4 x 640 of K = 640 3.9 and 5.0.  With twice the threads, and so twice
// the limit, 1 x 5120 of K = 1280 took 5.9 (fewer CTAs an SM); with two chunks a half warp 2 x 4096 of K = 4096 9.0
// against 8.5.
bool fuse_tokens_i8(const LinearI8Plan& p, int64_t M, int64_t K) {
  return !p.pair && M <= LS_FUSED_TOKENS && M * ((K + 127) / 128) <= LS_FUSED_THREADS / 16;
}

// Whether na bytes from a and nb bytes from b share any.
bool may_overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

size_t rows_bytes(int64_t rows, int64_t width, int64_t ld, int type) {
  return ((size_t)(rows - 1) * (size_t)ld + (size_t)width) * dtype_size(type);
}

template <typename T>
svdq_status launch_fused_i8(int dev, const LinearI8Plan& p, LinearI8Args& a, const int8_t* Wq,
                            cudaStream_t s) {
  static std::atomic<bool> attr[kMaxDevices];
  CUtensorMap tm_w;
  if (!make_map_2d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, Wq, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.K, 128, 128))
    return SVDQ_ERR_CUDA;
  const int per = code_chunks(a.K, p.split);
  a.nt = LS_FUSED_TOKENS;
  a.stages = std::min(per, 6);
  constexpr int most = 6 * LS_A_BYTES + LS_FUSED_THREADS / 16 * LS_FUSED_CHUNK + LS_TAIL_BYTES + 1024;
  const size_t smem = (size_t)a.stages * LS_A_BYTES + per * LS_FUSED_CHUNK + LS_TAIL_BYTES + 1024;
  svdq_status st;
  if ((st = allow_smem(k_linear_i8_split<T>, dev, attr, most)) != SVDQ_OK) return st;
  if (launch_pdl(k_linear_i8_split<T>, dim3((unsigned)(((int64_t)a.N + 127) / 128 * p.split)), dim3(LS_FUSED_THREADS), smem, s,
                 p.split, tm_w, tm_w, a, p.split) != cudaSuccess)
    return launch_failed();
  return launch_status();
}

// w_early: the kernel before this one on the stream is a quantizer of this library, which has waited for
// everything before it, so the weight may be read while it still runs.
svdq_status launch_linear_i8(int dev, DevInfo* d, const int8_t* Xq, const float* sx, const int8_t* Wq,
                             const float* sw, const float* bias, void* Y, int y_type, int64_t ldy, int64_t M,
                             int64_t N, int64_t K, int w_early, cudaStream_t s) {
  const LinearI8Plan p = plan_linear_i8(M, N, K, d->sms);
  LinearI8Args a = {};
  a.sx = sx;
  a.sw = sw;
  a.bias = bias;
  a.Y = Y;
  a.y_type = y_type;
  a.y_vec = y_vector(Y, y_type, ldy);
  a.ldy = ldy;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.nt = p.nt;
  a.w_early = w_early;
  a.stages = 0;
  CUtensorMap tm_x, tm_w;
  if (!make_map_2d(&tm_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, Xq, (uint64_t)K, (uint64_t)M, (uint64_t)K, 128,
                   (uint32_t)(p.pair ? 128 : p.nt)) ||
      !make_map_2d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, Wq, (uint64_t)K, (uint64_t)N, (uint64_t)K, 128,
                   (uint32_t)(p.pair ? p.nt / 2 : 128)))
    return SVDQ_ERR_CUDA;
  svdq_status st;
  if (p.pair) {
    const int64_t tiles = (M + 255) / 256 * ((N + p.nt - 1) / p.nt);
    if (tiles > kMaxDim) return SVDQ_ERR_UNSUPPORTED_SHAPE;
    if ((st = allow_smem(k_linear_i8_pair, dev, g_pair_attr, LP_SMEM)) != SVDQ_OK) return st;
    const int64_t pairs = std::min<int64_t>(tiles, d->sms / 2);
    a.strips = p.strips;
    a.cut = (int)(p.strips > 1 ? tiles / pairs * pairs : tiles);
    CUtensorMap tm_s = tm_w;
    if (p.strips > 1 && !make_map_2d(&tm_s, CU_TENSOR_MAP_DATA_TYPE_UINT8, Wq, (uint64_t)K, (uint64_t)N, (uint64_t)K, 128,
                                     (uint32_t)(p.nt / p.strips / 2)))
      return SVDQ_ERR_CUDA;
    if (launch_pdl(k_linear_i8_pair, dim3((unsigned)(2 * pairs)), dim3(LP_THREADS), (size_t)LP_SMEM, s, 2, tm_x, tm_w,
                   tm_s, a) != cudaSuccess)
      return launch_failed();
    return launch_status();
  }
  // A ring of at most 100 KB: two CTAs fit an SM, so that the next kernel's start overlaps this one's end.
  const int stage = LS_A_BYTES + p.nt * 128;
  const int per = (int)(((K + 127) / 128 + p.split - 1) / p.split);
  a.stages = std::min(per, 100 * 1024 / stage);
  const size_t smem = (size_t)std::max(a.stages * stage, p.nt * 512) + LS_TAIL_BYTES + 1024;
  if ((st = allow_smem(k_linear_i8_split<int8_t>, dev, g_split_attr, 100 * 1024 + LS_TAIL_BYTES + 1024)) != SVDQ_OK) return st;
  if (launch_pdl(k_linear_i8_split<int8_t>, dim3((unsigned)((N + 127) / 128 * p.split), (unsigned)((M + p.nt - 1) / p.nt)),
                 dim3(LS_THREADS), smem, s, p.split, tm_w, tm_x, a, p.split) != cudaSuccess)
    return launch_failed();
  return launch_status();
}

// ------------------------------------------------------------- group norm ---
constexpr int64_t kMaxNormC = GN_MAX_C;
constexpr int64_t kMaxNormS = int64_t(1) << 30;   // row numbers a few blocks past the end stay in 32 bits

constexpr int64_t kNormBlocks = 148;      // one block an SM of a B200
constexpr int kNormSmem = 232448 - 2048;  // dynamic shared memory of k_group_norm, at most

struct NormPlan {
  bool one;                 // k_group_norm; else k_group_stats and k_group_apply
  int nv, rp1, l2, rp2, threads1, threads2, P, rows;
};
NormPlan plan_norm(int64_t B, int64_t S, int64_t C, int64_t G, int row_bytes, bool quant) {
  NormPlan p;
  p.nv = (int)((C + 7) / 8);
  p.l2 = p.nv;
  if (quant) {                            // whole warps a row, or a power of two of lanes, at least four
    if (p.nv > 32) p.l2 = (p.nv + 31) / 32 * 32;
    else for (p.l2 = 4; p.l2 < p.nv;) p.l2 *= 2;
  }
  const bool large = !quant && B * S * row_bytes > (int64_t(16) << 20);
  const int most = large ? GN_MAX_THREADS : GN_SMALL_THREADS;
  const auto split = [&](int64_t blocks, int most) {
    p.P = (int)std::max<int64_t>(1, blocks);
    p.rows = (int)((S + p.P - 1) / p.P);
    p.P = (int)((S + p.rows - 1) / p.rows);
    p.rp1 = std::min(std::max(1, most / p.nv), p.rows);
    p.rp2 = std::min(std::max(1, most / p.l2), p.rows);
    p.threads1 = (p.nv * p.rp1 + 31) / 32 * 32;
    p.threads2 = (p.l2 * p.rp2 + 31) / 32 * 32;
  };
  const int64_t step = std::max(1, GN_SMALL_THREADS / p.nv);       // rows a block takes at a time
  // One launch where a cluster of up to eight blocks holds a sample, at least two steps a block.  Where the samples alone
  // do not fill the GPU, only up to 64 KB a block: above that the many blocks of two launches win.
  int64_t P = 1;
  while (P < 8 && S >= 4 * P * step) P *= 2;
  split(P, GN_SMALL_THREADS);
  const int threads = std::max(p.threads1, p.threads2);
  const int64_t held = (int64_t)p.rows * row_bytes, room = kNormSmem - 4 * gn_fixed_floats((int)G, threads);
  p.one = held <= room && (held <= (64 << 10) || B * p.P >= kNormBlocks);
  if (p.one) {
    p.threads1 = p.threads2 = threads;
    return p;
  }
  // Otherwise as many blocks as the GPU holds at one time, over all samples, with about four rows a thread, and no
  // more than keep a sample's partials few enough for every block to merge them.
  split(std::min<int64_t>({kNormBlocks / B, S / (4 * step), 16384 / G}), most);
  return p;
}

size_t group_norm_workspace(int64_t B, int64_t S, int64_t C, int64_t G) {
  size_t need = 16;
  for (int bytes = 2; bytes <= 4; bytes += 2)
    for (int quant = 0; quant < 2; ++quant) {
      const NormPlan p = plan_norm(B, S, C, G, (int)((C + 7) / 8) * 8 * bytes, quant != 0);
      if (!p.one) need = std::max(need, (size_t)B * (size_t)G * (size_t)p.P * sizeof(float2));
    }
  return need;
}

struct NormArgs {
  const void* X;
  int type;
  int64_t ldx, B, S, C, G;
  const float *gamma, *beta;
  float eps;
  int act;
  void* Y;
  int64_t ldy;
  const float* inv_s;
  int8_t* Xq;
  float* sx;
  void* ws;
  size_t ws_bytes;
};

template <typename T, bool VEC, bool QUANT>
svdq_status launch_norm(int dev, const NormArgs& n, cudaStream_t s) {
  const int row_bytes = (int)((n.C + 7) / 8) * Elem<T>::kWords * 4;
  const NormPlan p = plan_norm(n.B, n.S, n.C, n.G, row_bytes, QUANT);
  GroupNormArgs a;
  a.X = n.X;
  a.ldx = n.ldx;
  a.S = (int)n.S;
  a.C = (int)n.C;
  a.G = (int)n.G;
  a.nv = p.nv;
  a.rp1 = p.rp1;
  a.l2 = p.l2;
  a.rp2 = p.rp2;
  a.P = p.P;
  a.rows = p.rows;
  a.part = static_cast<float2*>(n.ws);
  a.gamma = n.gamma;
  a.beta = n.beta;
  a.eps = n.eps;
  a.act = n.act;
  a.streaming = n.B * n.S * n.C * (int64_t)sizeof(T) > (int64_t(48) << 20);
  // Of a tensor that L2 cannot hold, each block's last rows are kept there for the second pass, 64 MB over all blocks (a
  // megapixel of 128 channels 137 us, 144 without; 100 MB: 139).
  const int64_t total = n.B * n.S * (int64_t)row_bytes, held = int64_t(64) << 20;
  const bool large = VEC && total > held;
  a.hot = large ? p.rows - (int)(p.rows * held / total) : 0;
  a.Y = n.Y;
  a.ldy = n.ldy;
  a.inv_s = n.inv_s;
  a.Xq = n.Xq;
  a.sx = n.sx;
  const int64_t blocks = n.B * p.P;
  if (blocks > kMaxDim) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (p.one) {
    static std::atomic<bool> attr[kMaxDevices];
    const svdq_status st = allow_smem(k_group_norm<T, VEC, QUANT>, dev, attr, kNormSmem);
    if (st != SVDQ_OK) return st;
    const size_t smem = (size_t)gn_fixed_floats(a.G, p.threads1) * 4 + (size_t)p.rows * (size_t)row_bytes;
    if (launch_pdl(k_group_norm<T, VEC, QUANT>, dim3((unsigned)blocks), dim3(p.threads1), smem, s, p.P, a) != cudaSuccess)
      return launch_failed();
    return launch_status();
  }
  if (launch_pdl(large ? k_group_stats<T, VEC, VEC> : k_group_stats<T, VEC, false>, dim3((unsigned)blocks),
                 dim3(p.threads1), 0, s, 1, a) != cudaSuccess)
    return launch_failed();
  const size_t smem = ((size_t)n.G + 1) / 2 * 2 * sizeof(float2) + (size_t)p.threads2 * sizeof(GnMerge);
  if (launch_pdl(k_group_apply<T, VEC, QUANT>, dim3((unsigned)blocks), dim3(p.threads2), smem, s, 1, a) != cudaSuccess)
    return launch_failed();
  return launch_status();
}
template <typename T, bool QUANT>
svdq_status launch_norm(int dev, const NormArgs& n, cudaStream_t s) {
  const bool vec = n.C % 8 == 0 && n.ldx * sizeof(T) % 16 == 0 && (QUANT || n.ldy * sizeof(T) % 16 == 0);
  return vec ? launch_norm<T, true, QUANT>(dev, n, s) : launch_norm<T, false, QUANT>(dev, n, s);
}

template <bool QUANT>
svdq_status norm_impl(const NormArgs& n, cudaStream_t s) {
  if (n.B < 0 || n.S < 0 || n.C < 1 || n.G < 1 || !dtype_ok(n.type) || n.act < SVDQ_ACT_NONE ||
      n.act > SVDQ_ACT_GELU || !(n.eps >= 0.0f) || !std::isfinite(n.eps))
    return SVDQ_ERR_INVALID_ARG;
  if (n.C % n.G != 0 || n.C > kMaxNormC || (QUANT && n.C % 16 != 0) || n.B > kMaxDim || n.S > kMaxNormS ||
      (n.B > 0 && n.S > kMaxDim / n.B))
    return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (n.B == 0 || n.S == 0) return SVDQ_OK;        // an empty batch: nothing to launch
  svdq_status st = check_rows(n.X, n.type, n.C, n.ldx, false);
  if (st != SVDQ_OK) return st;
  if (QUANT) {
    if (!n.Xq || !n.sx) return SVDQ_ERR_INVALID_ARG;
    if (!aligned16(n.Xq) || !aligned16(n.sx) || (n.inv_s && !aligned16(n.inv_s))) return SVDQ_ERR_MISALIGNED;
  } else if ((st = check_rows(n.Y, n.type, n.C, n.ldy, false)) != SVDQ_OK) {
    return st;
  }
  if (!n.ws || n.ws_bytes < group_norm_workspace(n.B, n.S, n.C, n.G)) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(n.ws) || (n.gamma && !aligned16(n.gamma)) || (n.beta && !aligned16(n.beta))) return SVDQ_ERR_MISALIGNED;
  int dev;
  DevInfo* d;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  if (n.type == SVDQ_BF16) return launch_norm<__nv_bfloat16, QUANT>(dev, n, s);
  if (n.type == SVDQ_FP16) return launch_norm<__half, QUANT>(dev, n, s);
  return launch_norm<float, QUANT>(dev, n, s);
}

}  // namespace

extern "C" {

const char* svdq_status_string(int status) {
  switch (status) {
    case SVDQ_OK: return "SVDQ_OK";
    case SVDQ_ERR_INVALID_ARG: return "SVDQ_ERR_INVALID_ARG";
    case SVDQ_ERR_UNSUPPORTED_SHAPE: return "SVDQ_ERR_UNSUPPORTED_SHAPE";
    case SVDQ_ERR_MISALIGNED: return "SVDQ_ERR_MISALIGNED";
    case SVDQ_ERR_CUDA: return "SVDQ_ERR_CUDA";
    case SVDQ_ERR_TIMEOUT: return "SVDQ_ERR_TIMEOUT";
    case SVDQ_ERR_DEVICE: return "SVDQ_ERR_DEVICE";
    case SVDQ_ERR_SCRATCH: return "SVDQ_ERR_SCRATCH";
    case SVDQ_ERR_CHECK: return "SVDQ_ERR_CHECK";
    default: return "SVDQ_ERR_UNKNOWN";
  }
}

int svdq_version(void) { return 100; }

size_t svdq_sf_bytes(int64_t rows, int64_t K) {
  if (rows < 0 || K < 0 || K % 64 != 0) return 0;
  return (size_t)pad128(rows) * (size_t)(K / 16);
}

svdq_status svdq_pack_weight(const float* R, const uint16_t* L2b, int64_t K, int64_t N, int r, uint8_t* Wq,
                             uint8_t* SFw, float* gs_w, float* gs_w_host, uint16_t* L2p, svdq_stream_t stream) {
  svdq_status st = check_shape(1, N, K, r);
  if (st != SVDQ_OK) return st;
  if (!R || !Wq || !SFw || !gs_w || (r > 0 && (!L2b || !L2p))) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(R) || !aligned16(Wq) || !aligned16(SFw) || (r > 0 && (!aligned16(L2b) || !aligned16(L2p))))
    return SVDQ_ERR_MISALIGNED;
  int dev;
  DevInfo* d;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  unsigned int* bits = reinterpret_cast<unsigned int*>(gs_w);
  k_zero_u32<<<1, 1, 0, s>>>(bits);
  const int64_t n = K * N;
  int64_t blocks = (n / 4 + 255) / 256;
  if (blocks > 4 * (int64_t)d->sms) blocks = 4 * (int64_t)d->sms;
  if (blocks < 1) blocks = 1;
  k_absmax_f32<<<(unsigned)blocks, 256, 0, s>>>(R, n, bits);
  k_global_scale<<<1, 1, 0, s>>>(gs_w);
  const int64_t Npad = pad128(N);
  k_pack_weight<<<dim3((unsigned)(Npad / 128), (unsigned)(K / 64)), 128, 0, s>>>(R, (int)K, (int)N, (int)Npad, gs_w,
                                                                                  Wq, SFw);
  if (r > 0) k_layout_l2<<<(unsigned)((N + 127) / 128), 128, 0, s>>>(L2b, (int)N, r, L2p);
  if ((st = launch_status()) != SVDQ_OK) return st;
  if (gs_w_host) {
    if (cudaMemcpyAsync(gs_w_host, gs_w, sizeof(float), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
      return SVDQ_ERR_CUDA;
  }
  return SVDQ_OK;
}

size_t svdq_mx_sf_bytes(int64_t rows, int64_t K) {
  if (rows < 0 || K < 0 || K % 128 != 0) return 0;
  return (size_t)pad128(rows) * (size_t)(K / 32);
}

svdq_status svdq_pack_weight_mx(const float* R, const uint16_t* L2b, int64_t K, int64_t N, int r, uint8_t* Wq,
                                uint8_t* SFw, uint16_t* L2p, svdq_stream_t stream) {
  svdq_status st = check_shape(1, N, K, r);
  if (st != SVDQ_OK) return st;
  if (K % 128 != 0) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (!R || !Wq || !SFw || (r > 0 && (!L2b || !L2p))) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(R) || !aligned16(Wq) || !aligned16(SFw) || (r > 0 && (!aligned16(L2b) || !aligned16(L2p))))
    return SVDQ_ERR_MISALIGNED;
  int dev;
  DevInfo* d;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t Npad = pad128(N);
  k_pack_weight_mx<<<dim3((unsigned)(Npad / 128), (unsigned)(K / 128)), 128, 0, s>>>(R, (int)K, (int)N, (int)Npad,
                                                                                     Wq, SFw);
  if (r > 0) k_layout_l2<<<(unsigned)((N + 127) / 128), 128, 0, s>>>(L2b, (int)N, r, L2p);
  return launch_status();
}

svdq_status svdq_quantize_act_mx(const uint16_t* X, int64_t M, int64_t K, const float* inv_s, const uint16_t* L1fT,
                                 int r, float lr_scale, uint8_t* Xq, uint8_t* SFx, uint16_t* LAs, void* workspace,
                                 size_t workspace_bytes, svdq_stream_t stream) {
  svdq_status st = check_shape(M, 16, K, r);
  if (st != SVDQ_OK) return st;
  if (K % 128 != 0) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return SVDQ_OK;                 // an empty batch: nothing to launch
  if (!X || !inv_s || !Xq || !SFx || (r > 0 && (!L1fT || !LAs))) return SVDQ_ERR_INVALID_ARG;
  if (r > 0 && (!workspace || workspace_bytes < qa_workspace_bytes(M, r))) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(inv_s) || !aligned16(Xq) || !aligned16(SFx) ||
      (r > 0 && (!aligned16(L1fT) || !aligned16(LAs) || !aligned16(workspace))))
    return SVDQ_ERR_MISALIGNED;
  int dev;
  DevInfo* d;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  return dispatch_qa<true, true>(d, r, X, M, K, inv_s, 1.0f, L1fT, lr_scale, Xq, SFx, LAs, workspace,
                                 reinterpret_cast<cudaStream_t>(stream));
}

svdq_status svdq_linear_mx(const uint8_t* Xq, const uint8_t* SFx, const uint8_t* Wq, const uint8_t* SFw,
                           const uint16_t* LAs, const uint16_t* L2p, int r, const uint16_t* bias, void* Y, int y_fp32,
                           int64_t M, int64_t N, int64_t K, svdq_stream_t stream) {
  return linear_impl(Xq, SFx, 1.0f, Wq, SFw, 1.0f, LAs, L2p, r, bias, Y, y_fp32, M, N, K, 0, 0,
                     reinterpret_cast<cudaStream_t>(stream), 0, true);
}

size_t svdq_linear_gelu_quantize_workspace_bytes(int64_t M, int64_t N, int r2) {
  if (M < 1 || N < 1 || r2 < 0) return 0;
  return gq_workspace_bytes(M, N, r2);
}

svdq_status svdq_linear_gelu_quantize(const uint8_t* Xq, const uint8_t* SFx, float gs_x, const uint8_t* Wq,
                                      const uint8_t* SFw, float gs_w, const uint16_t* LAs, const uint16_t* L2p, int r,
                                      const uint16_t* bias, int64_t M, int64_t N, int64_t K, const float* inv_s2,
                                      float gs_x2, const uint16_t* L1fT2, int r2, float lr_scale2, uint8_t* Xq2,
                                      uint8_t* SFx2, uint16_t* LAs2, void* workspace, size_t workspace_bytes,
                                      svdq_stream_t stream) {
  svdq_status st = check_shape(M, N, K, r);
  if (st != SVDQ_OK) return st;
  if (N % 64 != 0 || (r2 != 0 && r2 != 16 && r2 != 32)) return SVDQ_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return SVDQ_OK;                 // an empty batch: nothing to launch
  if (r2 > 0 && workspace_bytes < gq_workspace_bytes(M, N, r2)) return SVDQ_ERR_INVALID_ARG;
  GqArgs g;
  g.inv_s2 = inv_s2;
  g.gs_x2 = gs_x2;
  g.L1fT2 = L1fT2;
  g.r2 = r2;
  g.lr_scale2 = lr_scale2;
  g.Xq2 = Xq2;
  g.SFx2 = SFx2;
  g.LAs2 = LAs2;
  g.part = static_cast<float*>(workspace);
  return linear_impl(Xq, SFx, gs_x, Wq, SFw, gs_w, LAs, L2p, r, bias, nullptr, 0, M, N, K, 0, 0,
                     reinterpret_cast<cudaStream_t>(stream), 0, false, &g);
}

svdq_status svdq_gelu_bf16(const uint16_t* X, int64_t n, uint16_t* Y, svdq_stream_t stream) {
  if (n < 0 || (n > 0 && (!X || !Y))) return SVDQ_ERR_INVALID_ARG;
  if (n == 0) return SVDQ_OK;
  if (!aligned16(X) || !aligned16(Y)) return SVDQ_ERR_MISALIGNED;
  int dev;
  DevInfo* d;
  svdq_status st;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  const int64_t nv = (n + 7) / 8;
  const int64_t cap = (int64_t)d->sms * 8;                   // 8 blocks of 256 threads per SM
  const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>((nv + 4 * 256 - 1) / (4 * 256), cap));
  if (launch_pdl(k_gelu_bf16, dim3(blocks), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), 1, X, n, Y) !=
      cudaSuccess)
    return SVDQ_ERR_CUDA;
  return launch_status();
}

svdq_status svdq_pack_weight_i8(const float* W_hat, int64_t K, int64_t N, int8_t* Wq, float* sw, svdq_stream_t stream) {
  svdq_status st = check_shape_i8(1, N, K);
  if (st != SVDQ_OK) return st;
  if (!W_hat || !Wq || !sw) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(W_hat) || !aligned16(Wq) || !aligned16(sw)) return SVDQ_ERR_MISALIGNED;
  int dev;
  DevInfo* d;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  k_pack_weight_i8<<<(unsigned)((N + 31) / 32), PW8_THREADS, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      W_hat, (int)K, (int)N, Wq, sw);
  return launch_status();
}

svdq_status svdq_quantize_act_i8(const void* X, int x_type, int64_t ldx, int64_t M, int64_t K, const float* inv_s,
                                 int8_t* Xq, float* sx, svdq_stream_t stream) {
  svdq_status st = check_shape_i8(M, 1, K);
  if (st != SVDQ_OK) return st;
  if (!dtype_ok(x_type)) return SVDQ_ERR_INVALID_ARG;
  if (M == 0) return SVDQ_OK;                 // an empty batch: nothing to launch
  if ((st = check_rows(X, x_type, K, ldx, true)) != SVDQ_OK) return st;
  if (!Xq || !sx) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(Xq) || !aligned16(sx) || (inv_s && !aligned16(inv_s))) return SVDQ_ERR_MISALIGNED;
  int dev;
  DevInfo* d;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  return launch_quantize_i8(d, X, x_type, ldx, M, K, inv_s, Xq, sx, reinterpret_cast<cudaStream_t>(stream));
}

svdq_status svdq_linear_i8(const int8_t* Xq, const float* sx, const int8_t* Wq, const float* sw, const float* bias,
                           void* Y, int y_type, int64_t ldy, int64_t M, int64_t N, int64_t K, svdq_stream_t stream) {
  svdq_status st = check_shape_i8(M, N, K);
  if (st != SVDQ_OK) return st;
  if (!dtype_ok(y_type)) return SVDQ_ERR_INVALID_ARG;
  if (M == 0) return SVDQ_OK;                 // an empty batch: nothing to launch
  if (!Xq || !sx || !Wq || !sw) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(Xq) || !aligned16(sx) || !aligned16(Wq) || !aligned16(sw) || (bias && !aligned16(bias)))
    return SVDQ_ERR_MISALIGNED;
  if ((st = check_rows(Y, y_type, N, ldy, false)) != SVDQ_OK) return st;
  int dev;
  DevInfo* d;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  return launch_linear_i8(dev, d, Xq, sx, Wq, sw, bias, Y, y_type, ldy, M, N, K, 0,
                          reinterpret_cast<cudaStream_t>(stream));
}

size_t svdq_forward_i8_workspace_bytes(int64_t M, int64_t K) {
  if (M < 1 || check_shape_i8(M, 1, K) != SVDQ_OK) return 0;
  return (size_t)M * (size_t)K + (size_t)M * sizeof(float);
}

svdq_status svdq_forward_i8(const void* X, int x_type, int64_t ldx, const float* inv_s, const int8_t* Wq,
                            const float* sw, const float* bias, void* Y, int y_type, int64_t ldy, int64_t M, int64_t N,
                            int64_t K, void* workspace, size_t workspace_bytes, svdq_stream_t stream) {
  svdq_status st = check_shape_i8(M, N, K);
  if (st != SVDQ_OK) return st;
  if (!dtype_ok(x_type) || !dtype_ok(y_type)) return SVDQ_ERR_INVALID_ARG;
  if (M == 0) return SVDQ_OK;                 // an empty batch: nothing to launch
  if ((st = check_rows(X, x_type, K, ldx, true)) != SVDQ_OK || (st = check_rows(Y, y_type, N, ldy, false)) != SVDQ_OK)
    return st;
  if (!Wq || !sw || !workspace || workspace_bytes < svdq_forward_i8_workspace_bytes(M, K)) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(Wq) || !aligned16(sw) || (bias && !aligned16(bias)) || (inv_s && !aligned16(inv_s)) ||
      !aligned16(workspace))
    return SVDQ_ERR_MISALIGNED;
  int dev;
  DevInfo* d;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int8_t* Xq = static_cast<int8_t*>(workspace);           // M x K codes (K % 16 == 0), then the M scales
  float* sx = reinterpret_cast<float*>(Xq + (size_t)M * (size_t)K);
  const LinearI8Plan p = plan_linear_i8(M, N, K, d->sms);
  // (One kernel for both reads X while it writes Y; the two kernels do not.)
  if (fuse_tokens_i8(p, M, K) && !may_overlap(X, rows_bytes(M, K, ldx, x_type), Y, rows_bytes(M, N, ldy, y_type))) {
    LinearI8Args a = {};
    a.sw = sw;
    a.bias = bias;
    a.Y = Y;
    a.y_type = y_type;
    a.y_vec = y_vector(Y, y_type, ldy);
    a.ldy = ldy;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.X = X;
    a.ldx = ldx;
    a.inv_s = inv_s;
    if (x_type == SVDQ_BF16) return launch_fused_i8<__nv_bfloat16>(dev, p, a, Wq, s);
    if (x_type == SVDQ_FP16) return launch_fused_i8<__half>(dev, p, a, Wq, s);
    return launch_fused_i8<float>(dev, p, a, Wq, s);
  }
  if ((st = launch_quantize_i8(d, X, x_type, ldx, M, K, inv_s, Xq, sx, s)) != SVDQ_OK) return st;
  return launch_linear_i8(dev, d, Xq, sx, Wq, sw, bias, Y, y_type, ldy, M, N, K, 1, s);
}

size_t svdq_group_norm_workspace_bytes(int64_t B, int64_t S, int64_t C, int64_t G) {
  if (B < 1 || S < 1 || C < 1 || G < 1 || C % G != 0 || C > kMaxNormC || B > kMaxDim || S > kMaxNormS || S > kMaxDim / B)
    return 0;
  return group_norm_workspace(B, S, C, G);
}

svdq_status svdq_group_norm(const void* X, int type, int64_t ldx, int64_t B, int64_t S, int64_t C, int64_t G,
                            const float* gamma, const float* beta, float eps, int act, void* Y, int64_t ldy,
                            void* workspace, size_t workspace_bytes, svdq_stream_t stream) {
  const NormArgs n = {X, type, ldx, B, S, C, G, gamma, beta, eps, act, Y, ldy, nullptr, nullptr, nullptr, workspace,
                      workspace_bytes};
  return norm_impl<false>(n, reinterpret_cast<cudaStream_t>(stream));
}

svdq_status svdq_group_norm_quantize_i8(const void* X, int type, int64_t ldx, int64_t B, int64_t S, int64_t C,
                                        int64_t G, const float* gamma, const float* beta, float eps, int act,
                                        const float* inv_s, int8_t* Xq, float* sx, void* workspace,
                                        size_t workspace_bytes, svdq_stream_t stream) {
  const NormArgs n = {X, type, ldx, B, S, C, G, gamma, beta, eps, act, nullptr, 0, inv_s, Xq, sx, workspace,
                      workspace_bytes};
  return norm_impl<true>(n, reinterpret_cast<cudaStream_t>(stream));
}

svdq_status svdq_call(int entry, const void* args) {
  if (!args) return SVDQ_ERR_INVALID_ARG;
  const unsigned char* words = static_cast<const unsigned char*>(args);   // at any alignment
  const auto word = [&](int i) {
    int64_t v;
    std::memcpy(&v, words + 8 * i, 8);
    return v;
  };
  const auto num = [&](int i) {              // an int parameter: a value outside its range is no valid argument
    const int64_t v = word(i);
    return v < INT32_MIN || v > INT32_MAX ? -1 : (int)v;
  };
  const auto real = [&](int i) {
    double v;
    std::memcpy(&v, words + 8 * i, 8);
    return (float)v;
  };
  const auto p = [&](int i) { return reinterpret_cast<void*>(word(i)); };
  const auto f = [&](int i) { return reinterpret_cast<float*>(word(i)); };
  const auto q = [&](int i) { return reinterpret_cast<int8_t*>(word(i)); };
  const auto stream = [&](int i) { return reinterpret_cast<svdq_stream_t>(word(i)); };
  switch (entry) {
    case SVDQ_CALL_QUANTIZE_ACT_I8:
      return svdq_quantize_act_i8(p(0), num(1), word(2), word(3), word(4), f(5), q(6), f(7), stream(8));
    case SVDQ_CALL_LINEAR_I8:
      return svdq_linear_i8(q(0), f(1), q(2), f(3), f(4), p(5), num(6), word(7), word(8), word(9), word(10), stream(11));
    case SVDQ_CALL_FORWARD_I8:
      return svdq_forward_i8(p(0), num(1), word(2), f(3), q(4), f(5), f(6), p(7), num(8), word(9), word(10), word(11),
                             word(12), p(13), (size_t)word(14), stream(15));
    case SVDQ_CALL_GROUP_NORM:
      return svdq_group_norm(p(0), num(1), word(2), word(3), word(4), word(5), word(6), f(7), f(8), real(9), num(10),
                             p(11), word(12), p(13), (size_t)word(14), stream(15));
    case SVDQ_CALL_GROUP_NORM_QUANTIZE_I8:
      return svdq_group_norm_quantize_i8(p(0), num(1), word(2), word(3), word(4), word(5), word(6), f(7), f(8), real(9),
                                         num(10), f(11), q(12), f(13), p(14), (size_t)word(15), stream(16));
    default: return SVDQ_ERR_INVALID_ARG;
  }
}

svdq_status svdq_calib_absmax_cols(const uint16_t* X, int64_t M, int64_t K, float* amax_x, int accumulate,
                                   svdq_stream_t stream) {
  if (M < 0 || K < 8 || K % 8 != 0 || K >= (int64_t(1) << 31) || !amax_x || (M > 0 && !X) ||
      (accumulate != 0 && accumulate != 1))
    return SVDQ_ERR_INVALID_ARG;
  if ((M > 0 && !aligned16(X)) || (reinterpret_cast<uintptr_t>(amax_x) & 3u)) return SVDQ_ERR_MISALIGNED;
  int dev;
  DevInfo* d;
  svdq_status st;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!accumulate && cudaMemsetAsync(amax_x, 0, (size_t)K * sizeof(float), s) != cudaSuccess) return SVDQ_ERR_CUDA;
  if (M == 0) return launch_status();
  const int gx = (int)((K + 255) / 256);
  // enough row slices for about four blocks per SM
  const int64_t want = std::max<int64_t>(1, (int64_t)d->sms * 4 / gx);
  const int slices = (int)std::min<int64_t>(want, (M + 63) / 64);
  const int rows = (int)((M + slices - 1) / slices);
  k_absmax_cols<<<dim3(gx, (unsigned)((M + rows - 1) / rows)), 256, 0, s>>>(X, M, (int)K, rows, amax_x);
  return launch_status();
}

svdq_status svdq_calib_absmax_rows(const double* W, int64_t K, int64_t N, double* amax_w, svdq_stream_t stream) {
  if (K < 1 || N < 1 || K >= (int64_t(1) << 31) || !W || !amax_w) return SVDQ_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(W) | reinterpret_cast<uintptr_t>(amax_w)) & 7u) return SVDQ_ERR_MISALIGNED;
  int dev;
  DevInfo* d;
  svdq_status st;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  k_absmax_rows<<<(unsigned)K, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(W, N, amax_w);
  return launch_status();
}

svdq_status svdq_calib_smooth(const float* amax_x, const double* amax_w, int64_t K, double alpha, double* s,
                              float* inv_s, svdq_stream_t stream) {
  if (K < 1 || K >= (int64_t(1) << 31) || !amax_x || !amax_w || !s || !inv_s || !(alpha >= 0.0 && alpha <= 1.0))
    return SVDQ_ERR_INVALID_ARG;
  int dev;
  DevInfo* d;
  svdq_status st;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  k_smooth<<<(unsigned)((K + 255) / 256), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(amax_x, amax_w, (int)K,
                                                                                           alpha, s, inv_s);
  return launch_status();
}

svdq_status svdq_calib_scale_rows(const double* W, const double* s, int64_t K, int64_t N, double* W_hat,
                                  svdq_stream_t stream) {
  if (K < 1 || N < 1 || !W || !s || !W_hat) return SVDQ_ERR_INVALID_ARG;
  int dev;
  DevInfo* d;
  svdq_status st;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  const int64_t blocks = std::min<int64_t>((K * N + 255) / 256, (int64_t)d->sms * 16);
  k_scale_rows<<<(unsigned)blocks, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(W, s, K, N, W_hat);
  return launch_status();
}

svdq_status svdq_calib_act_amax(const uint16_t* X, int64_t M, int64_t K, const float* inv_s, float* amax,
                                int accumulate, svdq_stream_t stream) {
  if (M < 0 || K < 8 || K % 8 != 0 || K >= (int64_t(1) << 31) || !inv_s || !amax || (M > 0 && !X) ||
      (accumulate != 0 && accumulate != 1))
    return SVDQ_ERR_INVALID_ARG;
  if ((M > 0 && !aligned16(X)) || !aligned16(inv_s) || (reinterpret_cast<uintptr_t>(amax) & 3u))
    return SVDQ_ERR_MISALIGNED;
  int dev;
  DevInfo* d;
  svdq_status st;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!accumulate && cudaMemsetAsync(amax, 0, sizeof(float), s) != cudaSuccess) return SVDQ_ERR_CUDA;
  if (M == 0) return launch_status();
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((M * (K / 8) + 255) / 256, (int64_t)d->sms * 8));
  k_act_amax<<<(unsigned)blocks, 256, 0, s>>>(X, M, (int)K, inv_s, amax);
  return launch_status();
}

void svdq_map_cache_stats(uint64_t* hits, uint64_t* misses) {
  std::lock_guard<std::mutex> lk(g_map_mu);
  if (hits) *hits = g_map_hits;
  if (misses) *misses = g_map_misses;
}

svdq_status svdq_dequant_weight(const uint8_t* Wq, const uint8_t* SFw, const float* gs_w, int64_t K, int64_t N,
                                float* Rq, svdq_stream_t stream) {
  svdq_status st = check_shape(1, N, K, 0);
  if (st != SVDQ_OK) return st;
  if (!Wq || !SFw || !gs_w || !Rq) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(Wq) || !aligned16(SFw) || !aligned16(Rq)) return SVDQ_ERR_MISALIGNED;
  int dev;
  DevInfo* d;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  k_dequant_weight<<<dim3((unsigned)((N + 127) / 128), (unsigned)(K / 64)), 128, 0,
                     reinterpret_cast<cudaStream_t>(stream)>>>(Wq, SFw, gs_w, (int)K, (int)N, Rq);
  return launch_status();
}

size_t svdq_quantize_act_workspace_bytes(int64_t M, int64_t K, int r) {
  if (M < 1 || K < 64 || K % 64 != 0 || r < 0 || r % 16 != 0 || r > 128) return 0;
  return qa_workspace_bytes(M, r);
}

svdq_status svdq_quantize_act(const uint16_t* X, int64_t M, int64_t K, const float* inv_s, float gs_x,
                              const uint16_t* L1fT, int r, float lr_scale, uint8_t* Xq, uint8_t* SFx, uint16_t* LAs,
                              void* workspace, size_t workspace_bytes, svdq_stream_t stream) {
  svdq_status st = check_shape(M, 16, K, r);
  if (st != SVDQ_OK) return st;
  if (M == 0) return SVDQ_OK;                 // an empty batch: nothing to launch
  if (!X || !inv_s || !Xq || !SFx || (r > 0 && (!L1fT || !LAs))) return SVDQ_ERR_INVALID_ARG;
  if (r > 0 && (!workspace || workspace_bytes < qa_workspace_bytes(M, r))) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(inv_s) || !aligned16(Xq) || !aligned16(SFx) ||
      (r > 0 && (!aligned16(L1fT) || !aligned16(LAs) || !aligned16(workspace))))
    return SVDQ_ERR_MISALIGNED;
  int dev;
  DevInfo* d;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  return dispatch_qa<true>(d, r, X, M, K, inv_s, gs_x, L1fT, lr_scale, Xq, SFx, LAs, workspace,
                           reinterpret_cast<cudaStream_t>(stream));
}

svdq_status svdq_quantize_act_noalloc(const uint16_t* X, int64_t M, int64_t K, const float* inv_s, float gs_x,
                                      const uint16_t* L1fT, int r, float lr_scale, uint8_t* Xq, uint8_t* SFx,
                                      uint16_t* LAs, svdq_stream_t stream) {
  svdq_status st = check_shape(M, 16, K, r);
  if (st != SVDQ_OK) return st;
  if (M == 0) return SVDQ_OK;                 // an empty batch: nothing to launch
  if (!X || !inv_s || !Xq || !SFx || (r > 0 && (!L1fT || !LAs))) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(inv_s) || !aligned16(Xq) || !aligned16(SFx) ||
      (r > 0 && (!aligned16(L1fT) || !aligned16(LAs))))
    return SVDQ_ERR_MISALIGNED;
  int dev;
  DevInfo* d;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void* ws = nullptr;
  if (r > 0) {
    if (noalloc_scratch_need(M, K, r, d->sms) > kNoAllocScratchBytes) return SVDQ_ERR_SCRATCH;
    if ((st = noalloc_scratch(dev, d, &ws)) != SVDQ_OK) return st;
    // the row-block counters start at 0 (a call that ran out of time can leave them set)
    if (cudaMemsetAsync(ws, 0, qa_ticket_bytes(M), s) != cudaSuccess) return SVDQ_ERR_CUDA;
  }
  return dispatch_qa<true>(d, r, X, M, K, inv_s, gs_x, L1fT, lr_scale, Xq, SFx, LAs, ws, s);
}

svdq_status svdq_lowrank_down(const uint16_t* X, int64_t M, int64_t K, const uint16_t* L1fT, int r, float lr_scale,
                              uint16_t* LAs, void* workspace, size_t workspace_bytes, svdq_stream_t stream) {
  svdq_status st = check_shape(M, 16, K, r);
  if (st != SVDQ_OK) return st;
  if (M == 0) return r == 0 ? SVDQ_ERR_INVALID_ARG : SVDQ_OK;   // an empty batch: nothing to launch
  if (r == 0 || !X || !L1fT || !LAs || !workspace || workspace_bytes < qa_workspace_bytes(M, r))
    return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(L1fT) || !aligned16(LAs) || !aligned16(workspace)) return SVDQ_ERR_MISALIGNED;
  int dev;
  DevInfo* d;
  if ((st = current_device(&dev, &d)) != SVDQ_OK) return st;
  return dispatch_qa<false>(d, r, X, M, K, nullptr, 1.0f, L1fT, lr_scale, nullptr, nullptr, LAs, workspace,
                            reinterpret_cast<cudaStream_t>(stream));
}

svdq_status svdq_lowrank_up(const uint16_t* LAs, const uint16_t* L2p, int r, float gs, void* Y, int y_fp32,
                            int64_t M, int64_t N, svdq_stream_t stream) {
  return linear_impl(nullptr, nullptr, 1.0f, nullptr, nullptr, gs, LAs, L2p, r, nullptr, Y, y_fp32, M, N, 0, 0, 0,
                     reinterpret_cast<cudaStream_t>(stream), 1);
}

svdq_status svdq_linear(const uint8_t* Xq, const uint8_t* SFx, float gs_x, const uint8_t* Wq, const uint8_t* SFw,
                        float gs_w, const uint16_t* LAs, const uint16_t* L2p, int r, const uint16_t* bias, void* Y,
                        int y_fp32, int64_t M, int64_t N, int64_t K, svdq_stream_t stream) {
  return linear_impl(Xq, SFx, gs_x, Wq, SFw, gs_w, LAs, L2p, r, bias, Y, y_fp32, M, N, K, 0, 0,
                     reinterpret_cast<cudaStream_t>(stream));
}

svdq_status svdq_linear_debug(const uint8_t* Xq, const uint8_t* SFx, float gs_x, const uint8_t* Wq,
                              const uint8_t* SFw, float gs_w, const uint16_t* LAs, const uint16_t* L2p, int r,
                              const uint16_t* bias, void* Y, int y_fp32, int64_t M, int64_t N, int64_t K,
                              int debug_flags, uint64_t timeout_ns, svdq_stream_t stream) {
#ifdef SVDQ_CHECK
  if (debug_flags & ~(LN_DBG_NO_LOADS | LN_DBG_MISALIGN)) return SVDQ_ERR_INVALID_ARG;
#else
  if (debug_flags & ~LN_DBG_NO_LOADS) return SVDQ_ERR_INVALID_ARG;   // the misaligned box only where checked
#endif
  return linear_impl(Xq, SFx, gs_x, Wq, SFw, gs_w, LAs, L2p, r, bias, Y, y_fp32, M, N, K, debug_flags, timeout_ns,
                     reinterpret_cast<cudaStream_t>(stream));
}

svdq_status svdq_get_device_error(svdq_stream_t stream, int* site) {
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return SVDQ_ERR_CUDA;
  unsigned int flags = 0, where = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&flags, svdq::g_err_flags, sizeof(flags)) != cudaSuccess ||
      cudaMemcpyFromSymbol(&where, svdq::g_err_site, sizeof(where)) != cudaSuccess ||
      cudaMemcpyToSymbol(svdq::g_err_flags, &zero, sizeof(zero)) != cudaSuccess ||
      cudaMemcpyToSymbol(svdq::g_err_site, &zero, sizeof(zero)) != cudaSuccess)
    return SVDQ_ERR_CUDA;
  if (site) *site = (int)where;
  if (flags & svdq::ERR_CHECK) return SVDQ_ERR_CHECK;
  return (flags & svdq::ERR_TIMEOUT) ? SVDQ_ERR_TIMEOUT : SVDQ_OK;
}

int svdq_build_flags(void) {
#ifdef SVDQ_CHECK
  return 1;
#else
  return 0;
#endif
}

}  // extern "C"
