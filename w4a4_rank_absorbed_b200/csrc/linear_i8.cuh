// Int8 GEMM with scales per token and channel:
//   Y[m, n] = f32(f32(acc) sx[m]) sw[n] + bias[n],  acc = sum_k Xq[m, k] Wq[n, k]  (int32, exact for K < 2^17)
// one fused multiply-add for the last product and the bias, rounded once to the type of Y.
//
// Both kernels run tcgen05.mma.kind::i8 on 128-byte chunks of K that TMA lands in 128-byte swizzled
// tiles (chunks past K and rows past M or N are zero-filled and add nothing).
#pragma once
#include <type_traits>

#include "int8.cuh"
#include "tc_i8.cuh"

namespace svdq {

constexpr uint64_t L8_TIMEOUT_NS = 2000000000ull;

struct LinearI8Args {
  const float* sx;
  const float* sw;
  const float* bias;
  void* Y;
  int y_type;
  int y_vec;            // Y's rows start on 16 bytes (2: on 32): vector stores
  int64_t ldy;
  int M, N, K;
  int nt;               // columns (pair kernel) or tokens (split kernel) of a tile
  int cut, strips;      // pair kernel: tiles from `cut` on are taken in `strips` strips of columns each
  int stages;           // ring slots (split kernel)
  int w_early;          // split kernel: the weight may be read before griddepcontrol.wait
  const void* X;        // split kernel that quantizes its tokens itself: their rows and smoothing factors
  int64_t ldx;
  const float* inv_s;
};

SVDQ_DEV float i8_dequant(int acc, float sx, float sw, float bias) {
  return __fmaf_rn(__fmul_rn(__int2float_rn(acc), sx), sw, bias);
}
SVDQ_DEV uint32_t pack_16(float lo, float hi, int type) {
  if (type == DT_BF16) return pack_bf16x2(lo, hi);
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
SVDQ_DEV void store_y(void* Y, int type, int64_t at, float y) {
  if (type == DT_BF16) static_cast<__nv_bfloat16*>(Y)[at] = __float2bfloat16_rn(y);
  else if (type == DT_FP16) static_cast<__half*>(Y)[at] = __float2half_rn(y);
  else static_cast<float*>(Y)[at] = y;
}

// ------------------------------------------------------------------ pair kernel ---
// Many tokens: persistent CTA pairs (one CTA an SM), tiles of 256 tokens x nt channels (nt a multiple of 32,
// 64..256), each CTA holding 128 of the tokens and half of the channels' codes in a 6-slot ring of 32 KB, and the
// sums of its 128 tokens in TMEM twice over (columns 0 and 256), so that a tile's epilogue runs under the next tile's
// MMAs.  A pair's MMA reads each operand byte from shared memory half as often as two CTAs' own would, and each CTA
// copies half of B.
// Bound by the tensor pipe, and in long runs by the power limit: 4608 x 4096 of K = 12288 138 us (3.36 POP/s), 4608 x
// 12288 of K = 4096 143, 4096 cubed 46.3; the pipe is busy 82 % of the active cycles at 4608 x 4096 of K = 4096.
// Narrow outputs are bound by the stores and by the last wave: 16384 x 320 of K = 320 8.6 us, 8192 x 1280 of K = 1280
// 16.7 (steps of 64 in nt: 9.2 and 18.4).  Roles are walked by whole warps that elect a lane for each copy and MMA:
// with one lane in a divergent branch a ring slot took 600 cycles to issue.
//   warp 0      copies: A and B boxes, both CTAs counting on the leader's barrier
//   warp 1      leader only: MMAs;  in both: TMEM
//   warps 4-11  epilogue: TMEM -> registers, scales and bias, stores (two warps a lane quarter)
constexpr int LP_STAGES = 6;
constexpr int LP_A_BYTES = 128 * 128;
constexpr int LP_STAGE_BYTES = 2 * LP_A_BYTES;
constexpr int LP_THREADS = 384;
constexpr int LP_EPI_WARP0 = 4;
constexpr int LP_EPI_WARPS = 8;
constexpr int LP_STG_BYTES = 2048 + 1024;        // a warp's 16 x 32 staging tile; its 128 channels' scales and biases
constexpr int LP_OFF_STG = LP_STAGES * LP_STAGE_BYTES;
constexpr int LP_OFF_BAR = LP_OFF_STG + LP_EPI_WARPS * LP_STG_BYTES;
constexpr int LP_SMEM = LP_OFF_BAR + 256 + 1024;
static_assert(LP_SMEM <= 232448, "shared memory of a CTA");

constexpr int LP_RASTER = 8;                             // 4, 12 and 16 measured no better
// Tiles run in groups of LP_RASTER row blocks, the row block fastest: the pairs at work at one time
// share few rows of X and few of Wq, which stay in L2.
SVDQ_DEV void pair_tile(int t, int num_m, int num_n, int& mb, int& nb) {
  const int per_group = LP_RASTER * num_n;
  const int first = t / per_group * LP_RASTER;
  const int gm = min(LP_RASTER, num_m - first);
  const int w = t % per_group;
  mb = first + w % gm;
  nb = w / gm;
}

// What a pair does at a time: columns col.. (w of them) of row block mb.  The tiles before a.cut fill whole rounds of
// all pairs; the last round's, where they are few, come in strips, so that more pairs share them.
struct PairWork {
  int mb, col, w;
};
SVDQ_DEV PairWork pair_work(const LinearI8Args& a, int i, int num_m, int num_n) {
  const bool whole = i < a.cut;
  const int tile = whole ? i : a.cut + (i - a.cut) / a.strips;
  PairWork p;
  int nb;
  pair_tile(tile, num_m, num_n, p.mb, nb);
  p.w = whole ? a.nt : a.nt / a.strips;
  p.col = nb * a.nt + (whole ? 0 : (i - a.cut) % a.strips * p.w);
  return p;
}

// 32 columns from n0 of one row a lane: rows row0 + lane (below a.M), sums v.  chan: the columns' scales, and
// 512 bytes on their biases, in shared memory.
SVDQ_DEV void store_chunk(const LinearI8Args& a, const uint32_t (&v)[32], int row0, int n0, float sx, uint32_t chan,
                          float* stg) {
  const int lane = threadIdx.x & 31;
  const int row = row0 + lane;
  if (n0 >= a.N || row0 >= a.M) return;                             // warp-uniform
  if (a.y_vec && n0 + 32 <= a.N) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float y[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 s = lds_v4(chan + 64 * h + 16 * i), b = lds_v4(chan + 512 + 64 * h + 16 * i);
        const int j = 16 * h + 4 * i;
        y[4 * i] = i8_dequant((int)v[j], sx, __uint_as_float(s.x), __uint_as_float(b.x));
        y[4 * i + 1] = i8_dequant((int)v[j + 1], sx, __uint_as_float(s.y), __uint_as_float(b.y));
        y[4 * i + 2] = i8_dequant((int)v[j + 2], sx, __uint_as_float(s.z), __uint_as_float(b.z));
        y[4 * i + 3] = i8_dequant((int)v[j + 3], sx, __uint_as_float(s.w), __uint_as_float(b.w));
      }
      if (row >= a.M) continue;
      const int64_t at = (int64_t)row * a.ldy + n0 + 16 * h;
      if (a.y_type == DT_FP32) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.Y) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
      } else {
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = pack_16(y[2 * i], y[2 * i + 1], a.y_type);
        uint16_t* dst = static_cast<uint16_t*>(a.Y) + at;
        if (a.y_vec == 2) {
          st_global_v8(dst, o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7]);
        } else {
          reinterpret_cast<uint4*>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
          reinterpret_cast<uint4*>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
    }
    return;
  }
  // Ragged columns or rows at any alignment: 16 rows at a time are turned in the warp's staging buffer (element
  // (r, c) at 32 r + (c ^ r): no bank conflict either way), and 32 lanes store a row's 32 columns.
  const int n = n0 + lane;
  const float s = lds_f32(chan + 4 * lane), b = lds_f32(chan + 512 + 4 * lane);
#pragma unroll 1
  for (int g = 0; g < 32; g += 16) {
    __syncwarp();
    if ((lane & 16) == g) {
#pragma unroll
      for (int j = 0; j < 32; ++j) stg[(lane & 15) * 32 + (j ^ (lane & 15))] = __fmul_rn(__int2float_rn((int)v[j]), sx);
    }
    __syncwarp();
    const int rows = min(16, a.M - row0 - g);
    if (n < a.N) {
#pragma unroll 4
      for (int i = 0; i < rows; ++i)
        store_y(a.Y, a.y_type, (int64_t)(row0 + g + i) * a.ldy + n, __fmaf_rn(stg[i * 32 + (lane ^ i)], s, b));
    }
  }
}

__global__ void __launch_bounds__(LP_THREADS, 1) k_linear_i8_pair(
    const __grid_constant__ CUtensorMap tm_x,    // uint8 {K, M}, box {128, 128}, SW128
    const __grid_constant__ CUtensorMap tm_w,    // uint8 {K, N}, box {128, nt / 2}, SW128
    const __grid_constant__ CUtensorMap tm_s,    // the same with box {128, nt / strips / 2}
    const LinearI8Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + LP_OFF_BAR);   // leader's: both CTAs' boxes landed
  uint64_t* empty = full + LP_STAGES;                                 // own: slot consumed by the pair's MMAs
  uint64_t* acc_full = empty + LP_STAGES;                             // own, per accumulator
  uint64_t* acc_empty = acc_full + 2;                                 // leader's, per accumulator
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = (int)warp_uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = warp_uniform(cluster_rank());
  const int nkt = (a.K + 127) >> 7;
  const int num_m = (a.M + 255) >> 8, num_n = (a.N + a.nt - 1) / a.nt;
  const int total = a.cut + (num_m * num_n - a.cut) * a.strips, first = blockIdx.x >> 1, step = gridDim.x >> 1;
  const uint64_t tmo = L8_TIMEOUT_NS;

  if (threadIdx.x == 0) {
    for (int s = 0; s < LP_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * LP_EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_w);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();                       // both CTAs' barriers and TMEM exist
  tc_fence_after();
  const uint32_t tbase = warp_uniform(*tmem_slot);
  const uint32_t full0 = warp_uniform(map_to_rank(smem_u32(full), 0));
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------------ copies ---
    int s = 0, issued = 0;
    uint32_t phase = 1;
    bool ok = true;
    for (int t = first; t < total && ok; t += step) {
      const PairWork p = pair_work(a, t, num_m, num_n);
      const int ya = p.mb * 256 + (int)rank * 128, yb = p.col + (int)rank * (p.w / 2);
      const uint32_t bytes = 2 * (LP_A_BYTES + (uint32_t)(p.w / 2) * 128u);    // of both CTAs
      const CUtensorMap* tm_b = t < a.cut ? &tm_w : &tm_s;
      for (int kt = 0; kt < nkt; ++kt) {
        if (!mbar_wait_warp(&empty[s], phase, tmo, abort_flag, 0x501)) {
          ok = false;
          break;
        }
        uint8_t* dst = smem + s * LP_STAGE_BYTES;
        const uint32_t bar = full0 + 8u * (uint32_t)s;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
          if (SVDQ_CHECK_OK(ya >= 0 && yb >= 0 && (uint32_t)(dst - smem_raw) + LP_STAGE_BYTES <= dyn_smem_bytes(), 0x5c1)) {
            tma_load_2d_pair(dst, &tm_x, bar, kt * 128, ya);
            tma_load_2d_pair(dst + LP_A_BYTES, tm_b, bar, kt * 128, yb);
          }
        }
        __syncwarp();
        ++issued;
        if (++s == LP_STAGES) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
    if (*abort_flag && rank == 0 && lane == 0) {
      // Give the copies in flight (both CTAs') the chance to land before the CTAs exit.
      int never = 0;
      for (int i = max(0, issued - LP_STAGES); i < issued; ++i)
        mbar_wait(&full[i % LP_STAGES], (uint32_t)((i / LP_STAGES) & 1), tmo, &never, 0x502);
    }
  } else if (warp == 1 && rank == 0) {
    // -------------------------------------------------------------------- MMAs ---
    const uint64_t desc0 = sdesc_kmajor_sw128(smem_u32(smem));
    int s = 0, n = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += step, ++n) {
      const uint32_t idesc = idesc_i8(256, t < a.cut ? a.nt : a.nt / a.strips);
      const uint32_t d = tbase + 256u * (uint32_t)(n & 1);
      if (n >= 2 && !mbar_wait_warp(&acc_empty[n & 1], (uint32_t)(((n >> 1) - 1) & 1), tmo, abort_flag, 0x511)) break;
      tc_fence_after();
      for (int kt = 0; kt < nkt; ++kt) {
        if (!mbar_wait_warp(&full[s], phase, tmo, abort_flag, 0x512)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t ad = desc0 + (uint64_t)(s * (LP_STAGE_BYTES / 16)), bd = ad + LP_A_BYTES / 16;
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 4; ++j) tc_mma_i8_pair(d, ad + 2 * j, bd + 2 * j, idesc, (kt | j) != 0 ? 1u : 0u);
          tc_commit_pair(&empty[s]);
          if (kt == nkt - 1) tc_commit_pair(&acc_full[n & 1]);
        }
        __syncwarp();
        if (++s == LP_STAGES) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
    if (*abort_flag) {
      int never = 0;
      if (elect_one()) tc_commit_pair(drain);
      __syncwarp();
      mbar_wait(drain, 0, tmo, &never, 0x513);
    }
  } else if (warp >= LP_EPI_WARP0) {
    // ---------------------------------------------------------------- epilogue ---
    const int ew = warp - LP_EPI_WARP0, q = warp & 3, h = ew >> 2;
    float* stg = reinterpret_cast<float*>(smem + LP_OFF_STG + ew * LP_STG_BYTES);
    float* chan = stg + 512;
    int n = 0;
    for (int t = first; t < total; t += step, ++n) {
      const PairWork p = pair_work(a, t, num_m, num_n);
      const int last = (((p.w >> 5) - 1 - h) & ~1) + h;  // this warp's 32-column chunks: h, h + 2, .. last
      const int row0 = p.mb * 256 + (int)rank * 128 + 32 * q, col0 = p.col + 32 * h;
      const float sx = row0 + lane < a.M ? __ldg(a.sx + row0 + lane) : 0.0f;
      __syncwarp();                                      // the last tile's reads of them are done
      // the tile's channel scales and biases, while the sums are on their way
      if (h + 2 * (lane >> 3) <= last) {                 // four columns a lane
        const int c = col0 + 64 * (lane >> 3) + 4 * (lane & 7);
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f), b = s;
        if (c + 4 <= a.N) {
          s = __ldg(reinterpret_cast<const float4*>(a.sw + c));
          if (a.bias) b = __ldg(reinterpret_cast<const float4*>(a.bias + c));
        } else {
          float* sv = reinterpret_cast<float*>(&s);
          float* bv = reinterpret_cast<float*>(&b);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + i < a.N) {
              sv[i] = __ldg(a.sw + c + i);
              if (a.bias) bv[i] = __ldg(a.bias + c + i);
            }
        }
        *reinterpret_cast<float4*>(chan + 4 * lane) = s;
        *reinterpret_cast<float4*>(chan + 128 + 4 * lane) = b;
      }
      __syncwarp();
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&acc_full[n & 1], (uint32_t)((n >> 1) & 1), tmo, abort_flag, 0x521))) break;
      tc_fence_after();
      const uint32_t ta = tbase + 256u * (uint32_t)(n & 1) + ((uint32_t)(32 * q) << 16);
      for (int c = h; c <= last; c += 2) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(ta + 32 * c, v);
        tmem_ld_wait();
        reg_fence(v);
        if (c == last) {                                 // all of this tile's sums are in registers: release it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(&acc_empty[n & 1]), 0));
        }
        store_chunk(a, v, row0, p.col + 32 * c, sx, smem_u32(chan) + 64u * (uint32_t)(c - h), stg);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();                       // neither CTA leaves while the other may still reach it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, 512);
  }
}

// ----------------------------------------------------------------- split kernel ---
// Few tokens, where the weight's bytes count: the roles of the operands are swapped (A = 128 channels of
// Wq, B = the tokens, nt of them), and the CTAs of a cluster share a tile's K axis, so that the GPU is
// full whatever N is.  Each CTA streams its K range through a ring, leaves its integer sums in shared
// memory, and after a cluster barrier sums a share of the tile's outputs over the cluster's CTAs (integers:
// the order does not matter).
// Bound by the weight's bytes where it is large (1 x 12288 of K = 4096 11.4 us, 50 MB: 0.68 of the copy bandwidth,
// 3.5 us of it launch, first loads and reduction), else by those latencies (1 x 4096 of K = 4096 from L2 4.8 us).
//   warp 0  copies, warp 1 MMAs and TMEM;  then all warps the epilogue
// TMEM: CTAs of several such kernels may share an SM, and one that waits for columns while its cluster waits for it
// must not meet another in the same position.  With a cluster a CTA has at least two ring slots, so at most six (nt
// 16..32: 32 columns each), four (33..80: 64 or 128) or three (81..128: 128) fit an SM's shared memory: 512 columns
// always do.
constexpr int LS_THREADS = 256;
constexpr int LS_A_BYTES = 128 * 128;
constexpr int LS_TAIL_BYTES = 256 + 1024;                 // barriers, then the tile's token scales

// One or a few tokens quantized by the GEMM itself (XT their type; int8_t: they come as codes): every CTA reads
// all of their rows for the maxima (from L2; sharing the maxima would take a cluster barrier), then writes
// the codes of its own K range where TMA would have put them, while the first weight boxes are on their way.  One
// launch instead of two.
constexpr int LS_FUSED_TOKENS = 16;                       // nt; a chunk of 128 of K is 16 rows of 128 bytes
constexpr int LS_FUSED_CHUNK = LS_FUSED_TOKENS * 128;
constexpr int LS_FUSED_THREADS = 512;
template <typename XT>
__host__ __device__ constexpr int split_threads() {
  return std::is_same<XT, int8_t>::value ? LS_THREADS : LS_FUSED_THREADS;
}
// All threads.  A half warp takes one of the rows' chunks of 128 columns, whose x_hat stays in registers between the
// maximum and the codes (with two or four, unrolled, the longer code alone cost 0.2 and 0.6 us where it had
// nothing to do).  top: zeroes; codes: the CTA's chunks, k_lo to k_hi.
template <typename T>
SVDQ_DEV void quantize_tokens(const LinearI8Args& a, int k_lo, int k_hi, uint32_t* top, float* sxs, uint8_t* codes) {
  const int nkt = (a.K + 127) >> 7, l = threadIdx.x & 15;
  const int unit = threadIdx.x >> 4, row = unit / nkt, chunk = unit - row * nkt, v = chunk * 16 + l;
  const bool in = row < a.M && 8 * v < a.K;
  uint32_t w[Elem<T>::kWords];
  float4 s0 = make_float4(1.f, 1.f, 1.f, 1.f), s1 = s0;
#pragma unroll
  for (int i = 0; i < Elem<T>::kWords; ++i) w[i] = 0u;
  if (in) load8(static_cast<const T*>(a.X) + (int64_t)row * a.ldx + 8 * v, w);
  if (in && a.inv_s) {
    s0 = __ldg(reinterpret_cast<const float4*>(a.inv_s) + 2 * v);
    s1 = __ldg(reinterpret_cast<const float4*>(a.inv_s) + 2 * v + 1);
  }
  float f[8], m = 0.0f;
  Elem<T>::unpack(w, f);
  const float2 xh[4] = {mul_f32x2(make_float2(f[0], f[1]), make_float2(s0.x, s0.y)),
                        mul_f32x2(make_float2(f[2], f[3]), make_float2(s0.z, s0.w)),
                        mul_f32x2(make_float2(f[4], f[5]), make_float2(s1.x, s1.y)),
                        mul_f32x2(make_float2(f[6], f[7]), make_float2(s1.z, s1.w))};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max_abs(m, xh[i].x, xh[i].y);
  uint32_t b = __float_as_uint(m);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) b = umax(b, __shfl_xor_sync(0xFFFFFFFFu, b, o));
  if (l == 0 && row < a.M) atomicMax(top + row, b);
  __syncthreads();
  if (row >= a.M) return;
  if (chunk == 0 && l == 0) sxs[row] = i8_scale_or_mul(top[row], true);
  if (chunk < k_lo || chunk >= k_hi) return;
  const float mul = i8_scale_or_mul(top[row], false);
  const uint2 c = i8_codes(xh, mul);
  *reinterpret_cast<uint2*>(codes + (chunk - k_lo) * LS_FUSED_CHUNK + row * 128 + ((((l >> 1) ^ row) & 7) << 4) +
                            8 * (l & 1)) = mul == 0.0f ? make_uint2(0u, 0u) : c;
}

// chunks of 128 of K that a CTA of a cluster of `split` has at most
__host__ __device__ __forceinline__ int code_chunks(int K, int split) { return (((K + 127) >> 7) + split - 1) / split; }

template <typename XT>
__global__ void __launch_bounds__(split_threads<XT>()) k_linear_i8_split(
    const __grid_constant__ CUtensorMap tm_w,    // uint8 {K, N}, box {128, 128}, SW128
    const __grid_constant__ CUtensorMap tm_x,    // uint8 {K, M}, box {128, nt}, SW128 (codes only)
    const LinearI8Args a, const int split) {
  constexpr bool CODES = std::is_same<XT, int8_t>::value;
  constexpr int THREADS = split_threads<XT>();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = LS_A_BYTES + (CODES ? a.nt * 128 : 0);
  const int ring = max(a.stages * stage_bytes, a.nt * 512);            // the sums take the ring's place
  // 16 tokens' codes of the CTA's K range lie past the ring where the kernel makes them
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + ring + (CODES ? 0 : code_chunks(a.K, split) * LS_FUSED_CHUNK));
  uint64_t* empty = full + a.stages;
  uint64_t* acc_full = empty + a.stages;
  uint64_t* drain = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* sxs = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(full) + 256);
  uint32_t* top = reinterpret_cast<uint32_t*>(sxs + 128);              // the tokens' largest magnitudes

  const int warp = (int)warp_uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rank = split > 1 ? (int)warp_uniform(cluster_rank()) : 0;
  const int nb = blockIdx.x / split, mb = blockIdx.y;
  const int nkt = (a.K + 127) >> 7;
  const int k_lo = (int)((int64_t)nkt * rank / split), k_hi = (int)((int64_t)nkt * (rank + 1) / split);
  const int nk = k_hi - k_lo;                                          // at least 1: split <= nkt
  const uint32_t cols = a.nt <= 32 ? 32u : a.nt <= 64 ? 64u : a.nt <= 128 ? 128u : 256u;
  const uint64_t tmo = L8_TIMEOUT_NS;

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_w);
    if (CODES) tma_prefetch_desc(&tm_x);
  }
  if (!CODES && threadIdx.x < LS_FUSED_TOKENS) top[threadIdx.x] = 0u;
  if (warp == 1) {
    tmem_alloc(tmem_slot, cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = warp_uniform(*tmem_slot);
  int issued = 0;                                                      // copying warp: ring rounds begun

  if (!CODES) griddep_wait();
  const int ahead = !CODES || a.w_early ? min(nk, a.stages) : 0;
  if (warp == 0) {
    const int yw = nb * 128;
    // The weight's first boxes may come before the wait where the kernel launched just before this one has
    // itself waited for all earlier work (svdq_forward_i8's quantizer): nothing in flight writes the weight.
    for (int kt = 0; kt < ahead; ++kt) {
      uint8_t* dst = smem + kt * stage_bytes;
      if (elect_one()) {
        mbar_arrive_expect_tx(&full[kt], (uint32_t)stage_bytes);
        if (SVDQ_CHECK_OK((uint32_t)(dst - smem_raw) + stage_bytes <= dyn_smem_bytes(), 0x5c2))
          tma_load_2d(dst, &tm_w, &full[kt], (k_lo + kt) * 128, yw);
      }
      __syncwarp();
    }
    issued = ahead;
  }
  if constexpr (!CODES) {
    griddep_launch_dependents();
    quantize_tokens<XT>(a, k_lo, k_hi, top, sxs, smem + ring);
    fence_proxy_async();                                                // the MMAs read the codes
    __syncthreads();
  }
  if (warp == 0) {
    const int yw = nb * 128, yx = mb * a.nt;
    if (CODES) griddep_wait();
    int s = 0;
    uint32_t phase = CODES ? 1 : 0;                                     // !CODES: from the ring's second round on
    for (int kt = CODES ? 0 : ahead; kt < nk; ++kt) {
      uint8_t* dst = smem + s * stage_bytes;
      if (kt >= ahead && !mbar_wait_warp(&empty[s], phase, tmo, abort_flag, 0x531)) break;
      if (elect_one()) {
        if (kt >= ahead) mbar_arrive_expect_tx(&full[s], (uint32_t)stage_bytes);
        if (SVDQ_CHECK_OK((uint32_t)(dst - smem_raw) + stage_bytes <= dyn_smem_bytes(), 0x5c3)) {
          if (kt >= ahead) tma_load_2d(dst, &tm_w, &full[s], (k_lo + kt) * 128, yw);
          if (CODES) tma_load_2d(dst + LS_A_BYTES, &tm_x, &full[s], (k_lo + kt) * 128, yx);
        }
      }
      __syncwarp();
      issued = max(issued, kt + 1);
      if (++s == a.stages) {
        s = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_i8(128, a.nt);
    const uint64_t desc0 = sdesc_kmajor_sw128(smem_u32(smem));
    int kt = 0, s = 0;
    uint32_t phase = 0;
    for (; kt < nk; ++kt) {
      if (!mbar_wait_warp(&full[s], phase, tmo, abort_flag, 0x532)) break;
      tc_fence_after();
      const uint64_t ad = desc0 + (uint64_t)(s * (stage_bytes / 16));
      const uint64_t bd = CODES ? ad + LS_A_BYTES / 16 : desc0 + (uint64_t)((ring + kt * LS_FUSED_CHUNK) / 16);
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < 4; ++j) tc_mma_i8(tbase, ad + 2 * j, bd + 2 * j, idesc, (kt | j) != 0 ? 1u : 0u);
        if (kt + a.stages < nk) tc_commit(&empty[s]);    // nobody waits for the last round of slots
        if (kt == nk - 1) tc_commit(acc_full);
      }
      __syncwarp();
      if (++s == a.stages) {
        s = 0;
        phase ^= 1u;
      }
    }
    if (kt < nk) {
      int never = 0;
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      mbar_wait(drain, 0, tmo, &never, 0x534);
    }
  }
  __syncwarp();

  // ------------------------------------------------------------------ epilogue ---
  if (CODES) {
    if (warp != 0) griddep_wait();                       // the copying warp has waited
    __syncwarp();
    griddep_launch_dependents();
  }
  const int tokens = min(a.nt, a.M - mb * a.nt);
  const int n = nb * 128 + 4 * lane;                     // four channels a lane
  float s4[4], b4[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s4[i] = n + i < a.N ? __ldg(a.sw + n + i) : 0.0f;
    b4[i] = a.bias && n + i < a.N ? __ldg(a.bias + n + i) : 0.0f;
  }
  if (CODES)
    for (int t = threadIdx.x; t < tokens; t += THREADS) sxs[t] = __ldg(a.sx + mb * a.nt + t);
  const bool got = __all_sync(0xFFFFFFFFu, mbar_wait(acc_full, 0, tmo, abort_flag, 0x533));
  if (!got && warp == 0 && lane == 0) {                  // let the copies in flight land before the CTA exits
    int never = 0;
    for (int kt = max(0, issued - a.stages); kt < issued; ++kt)
      mbar_wait(&full[kt % a.stages], (uint32_t)((kt / a.stages) & 1), tmo, &never, 0x535);
  }
  __syncwarp();
  tc_fence_after();
  // Every copy has landed and every MMA is done: the ring holds the sums now, nt rows (tokens) of 128 channels.
  int* part = reinterpret_cast<int*>(smem);
  const int q = warp & 3;
  if (got) {
    for (int c0 = 16 * (warp >> 2); c0 < a.nt; c0 += 32) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(tbase + ((uint32_t)(32 * q) << 16) + (uint32_t)c0, v);
      tmem_ld_wait();
      reg_fence16(v);
#pragma unroll
      for (int j = 0; j < 16; ++j) part[(c0 + j) * 128 + 32 * q + lane] = (int)v[j];
    }
  }
  tc_fence_before();
  if (split > 1) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, cols);
  }
  const uint32_t mine = smem_u32(part) + 16u * (uint32_t)lane;
#pragma unroll 4
  for (int t = rank + split * warp; t < tokens; t += split * (THREADS / 32)) {
    int4 acc = make_int4(0, 0, 0, 0);
    for (int r = 0; r < split; ++r) {
      const int4 v = split > 1 ? ld_cluster_v4(map_to_rank(mine + 512u * (uint32_t)t, (uint32_t)r))
                               : *reinterpret_cast<const int4*>(part + t * 128 + 4 * lane);
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
    const int row = mb * a.nt + t;
    const float sx = sxs[t];
    const float y0 = i8_dequant(acc.x, sx, s4[0], b4[0]), y1 = i8_dequant(acc.y, sx, s4[1], b4[1]);
    const float y2 = i8_dequant(acc.z, sx, s4[2], b4[2]), y3 = i8_dequant(acc.w, sx, s4[3], b4[3]);
    const int64_t at = (int64_t)row * a.ldy + n;
    if (a.y_vec && n + 4 <= a.N) {
      if (a.y_type == DT_FP32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.Y) + at) = make_float4(y0, y1, y2, y3);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.Y) + at) =
            make_uint2(pack_16(y0, y1, a.y_type), pack_16(y2, y3, a.y_type));
    } else {
      if (n < a.N) store_y(a.Y, a.y_type, at, y0);
      if (n + 1 < a.N) store_y(a.Y, a.y_type, at + 1, y1);
      if (n + 2 < a.N) store_y(a.Y, a.y_type, at + 2, y2);
      if (n + 3 < a.N) store_y(a.Y, a.y_type, at + 3, y3);
    }
  }
  __syncwarp();
  if (split > 1) cluster_sync_all();                     // no CTA leaves while another reads its sums
}

}  // namespace svdq
