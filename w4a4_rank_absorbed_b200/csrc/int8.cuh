// 8-bit integer form of the layer (SmoothQuant W8A8): the codec of weights and activations.
//
// "From SmoothQuant to SVDQuant", section Smooth Quant (W8A8): X diag(s)^-1 and diag(s) W are both
// quantized to 8-bit integers.  Scales are per row of the activations (token) and per column of the
// weight (output channel), so they leave the sum over K and the product of codes is an exact integer:
//   a  = max over the row of |x_hat|,  x_hat = f32(x * inv_s)
//   sx = f32(a / 127),  q = rint_even(f32(x_hat * f32(127 / a)))            (|q| <= 127)
//   a < 2^-100: sx = 0 and all codes 0 (127 / a would leave binary32's range for the smallest a);
//   a infinite or NaN: sx = NaN and all codes 0, so that the whole output row is NaN.
// Every step is one correctly rounded binary32 operation, so codes and scales are reproducible bit for bit.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace svdq {

enum : int { DT_BF16 = 0, DT_FP32 = 1, DT_FP16 = 2 };

// Element types: 8 consecutive elements are kWords 32-bit words.
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kWords = 4;
  SVDQ_DEV static void unpack(const uint32_t (&w)[4], float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  }
  SVDQ_DEV static void pack(const float (&f)[8], uint32_t (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  }
  SVDQ_DEV static float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
  SVDQ_DEV static __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
  static constexpr int kWords = 4;
  SVDQ_DEV static void unpack(const uint32_t (&w)[4], float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
  SVDQ_DEV static void pack(const float (&f)[8], uint32_t (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  SVDQ_DEV static float to_f32(__half v) { return __half2float(v); }
  SVDQ_DEV static __half from_f32(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<float> {
  static constexpr int kWords = 8;
  SVDQ_DEV static void unpack(const uint32_t (&w)[8], float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  }
  SVDQ_DEV static void pack(const float (&f)[8], uint32_t (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
  }
  SVDQ_DEV static float to_f32(float v) { return v; }
  SVDQ_DEV static float from_f32(float v) { return v; }
};

// Eight consecutive elements at `p` (16-byte aligned).
template <typename T>
SVDQ_DEV void load8(const T* p, uint32_t (&w)[Elem<T>::kWords]) {
#pragma unroll
  for (int i = 0; i < Elem<T>::kWords / 4; ++i) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
    w[4 * i] = v.x;
    w[4 * i + 1] = v.y;
    w[4 * i + 2] = v.z;
    w[4 * i + 3] = v.w;
  }
}

// |x| as an unsigned integer: the order of magnitudes, with infinities and NaN above every number.
SVDQ_DEV uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
SVDQ_DEV uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
// max(m, |a|, |b|) for m >= 0; NaN (as 0x7FFFFFFF) if any is.  Its bits order as abs_bits' do.
SVDQ_DEV float max_abs(float m, float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// Scale and multiplier of a row (or channel) whose largest magnitude has the bits `a`.
SVDQ_DEV void i8_scale(uint32_t a, float& scale, float& mul) {
  if (a >= 0x7F800000u) {                       // infinite or NaN
    scale = __uint_as_float(0x7FC00000u);
    mul = 0.0f;
  } else if (a < ((127u - 100u) << 23)) {       // below 2^-100
    scale = 0.0f;
    mul = 0.0f;
  } else {
    scale = __fdiv_rn(__uint_as_float(a), 127.0f);
    mul = __fdiv_rn(127.0f, __uint_as_float(a));
  }
}
// One of the two, by one division: lanes that need either then exchange them.
SVDQ_DEV float i8_scale_or_mul(uint32_t a, bool scale) {
  if (a >= 0x7F800000u) return scale ? __uint_as_float(0x7FC00000u) : 0.0f;
  if (a < ((127u - 100u) << 23)) return 0.0f;
  const float top = __uint_as_float(a);
  return __fdiv_rn(scale ? top : 127.0f, scale ? 127.0f : top);
}
// Code of x (0 whatever x is where mul = 0: an infinite x times 0 is NaN, which has no integer).
SVDQ_DEV int i8_code(float x, float mul) { return mul == 0.0f ? 0 : __float2int_rn(__fmul_rn(x, mul)); }
// Weight packing: W_hat (K x N float32, N contiguous) -> Wq (N x K codes), sw (N).  A block takes 32
// columns: its 16 warps walk the rows once for the column maxima (lane = column, 128-byte rows) and once
// more for the codes, turned through a shared tile of 128 rows so that Wq is written along K.
constexpr int PW8_THREADS = 512;
__global__ void __launch_bounds__(PW8_THREADS) k_pack_weight_i8(const float* __restrict__ W, int K, int N,
                                                                int8_t* __restrict__ Wq, float* __restrict__ sw) {
  __shared__ uint32_t part[16][32];
  __shared__ __align__(16) int8_t tile[32][128 + 16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = blockIdx.x * 32 + lane;
  const bool in = n < N;
  uint32_t a = 0u;
  if (in)
#pragma unroll 8
    for (int k = warp; k < K; k += 16) a = umax(a, abs_bits(__ldg(W + (int64_t)k * N + n)));
  part[warp][lane] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) a = umax(a, part[i][lane]);
  float scale, mul;
  i8_scale(a, scale, mul);
  if (warp == 0 && in) sw[n] = scale;
  const int wc = threadIdx.x >> 4, wk = (threadIdx.x & 15) * 8;      // column and bytes this thread writes
  for (int k0 = 0; k0 < K; k0 += 128) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = k0 + warp * 8 + i;
      tile[lane][warp * 8 + i] = (in && k < K) ? (int8_t)i8_code(__ldg(W + (int64_t)k * N + n), mul) : (int8_t)0;
    }
    __syncthreads();
    if (blockIdx.x * 32 + wc < N && k0 + wk < K)
      *reinterpret_cast<uint2*>(Wq + (int64_t)(blockIdx.x * 32 + wc) * K + k0 + wk) =
          *reinterpret_cast<const uint2*>(&tile[wc][wk]);
    __syncthreads();
  }
}

// Eight codes of x_hat as one byte each: f32(x_hat mul) plus 1.5 2^23 leaves rint of it (to even, as the sum is
// rounded to whole numbers) in the low bits of the sum, whose low byte is the code.  (Product and sum not as packed
// pairs: those came out as one fused operation, off at ties.)
SVDQ_DEV uint2 i8_codes(const float2 (&xh)[4], float mul) {
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[2 * i] = __float_as_uint(__fadd_rn(__fmul_rn(xh[i].x, mul), 12582912.0f));
    c[2 * i + 1] = __float_as_uint(__fadd_rn(__fmul_rn(xh[i].y, mul), 12582912.0f));
  }
  return make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410));
}
// The same of x_hat = f32(x s).
SVDQ_DEV uint2 i8_codes(const float (&x)[8], const float (&s)[8], float mul) {
  float2 xh[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    xh[i] = mul_f32x2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(s[2 * i], s[2 * i + 1]));
  return i8_codes(xh, mul);
}

// Activation quantization.  A group of threads, a warp or a block, owns a row at a time, each thread VPT vectors
// of 8 elements of it (vector j at its index + j times the group's size), the same columns in every row, so
// that their smoothing factors stay in registers; X is read once and held in registers between the maximum
// and the codes, and the group's next row is on its way while this one is reduced.
// HBM-bound for many rows (3 K bytes a 16-bit row).  Measured: 18432 x 4096 39.1 us, 0.90 of the copy
// bandwidth; 4608 x 4096 11.7 us, 0.75 (18.1 with four rows and 512 threads a block, whose registers left one
// block an SM); one row of 4096 1.6 us.  Up to 1024 columns a warp holds a row, without barriers (16384 x
// 320: 5.2 us, 5.8 with a block a row), unless the rows are too few to fill the GPU with warps (77 x 640: 1.9 us,
// 1.5 with a block); up to 16384 a block does; beyond that k_quantize_long_i8 reads rows twice.
constexpr int QI_MAX_THREADS = 512;
template <typename T, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : QI_MAX_THREADS) k_quantize_act_i8(
    const T* __restrict__ X, int64_t M, int K, int64_t ldx, const float* __restrict__ inv_s, int8_t* __restrict__ Xq,
    float* __restrict__ sx) {
  constexpr int W = Elem<T>::kWords;
  __shared__ uint32_t part[2][QI_MAX_THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int me = WARP ? lane : threadIdx.x, size = WARP ? 32 : blockDim.x;
  const int64_t step = WARP ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
  const int nv = K >> 3;
  // Everything earlier on the stream is done before this grid lets its dependent start (k_linear_i8_split's
  // early weight copies rest on that).
  griddep_wait();
  griddep_launch_dependents();
  float s[VPT][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = me + j * size;
#pragma unroll
    for (int i = 0; i < 8; ++i) s[j][i] = 1.0f;
    if (inv_s && v < nv) {
      const float4 s0 = __ldg(reinterpret_cast<const float4*>(inv_s) + 2 * v);
      const float4 s1 = __ldg(reinterpret_cast<const float4*>(inv_s) + 2 * v + 1);
      s[j][0] = s0.x; s[j][1] = s0.y; s[j][2] = s0.z; s[j][3] = s0.w;
      s[j][4] = s1.x; s[j][5] = s1.y; s[j][6] = s1.z; s[j][7] = s1.w;
    }
  }
  uint32_t w[VPT][W], nx[VPT][W];
  const auto fetch = [&](int64_t row, uint32_t(&d)[VPT][W]) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = me + j * size;
      if (v < nv && row < M) {
        load8(X + row * ldx + 8 * v, d[j]);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) d[j][i] = 0u;
      }
    }
  };
  int buf = 0;
  int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
  fetch(row, w);
  for (; row < M; row += step) {                         // uniform over the group
    fetch(row + step, nx);
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float f[8];
      Elem<T>::unpack(w[j], f);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 h = mul_f32x2(make_float2(f[i], f[i + 1]), make_float2(s[j][i], s[j][i + 1]));
        top = max_abs(top, h.x, h.y);
      }
    }
    uint32_t a = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top));
    if (!WARP) {
      if (lane == 0) part[buf][warp] = a;                // two buffers: one barrier a row
      __syncthreads();
      a = __reduce_max_sync(0xFFFFFFFFu, lane < (size >> 5) ? part[buf][lane] : 0u);
      buf ^= 1;
    }
    const float either = i8_scale_or_mul(a, lane == 0);  // lane 0 the scale, the others the multiplier
    if (me == 0) sx[row] = either;
    const float mul = __shfl_sync(0xFFFFFFFFu, either, 1);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = me + j * size;
      if (v < nv) {
        float f[8];
        Elem<T>::unpack(w[j], f);
        const uint2 c = i8_codes(f, s[j], mul);
        // where the multiplier is 0 the row has no codes (0 times an infinite element has none)
        *reinterpret_cast<uint2*>(Xq + row * K + 8 * v) = mul == 0.0f ? make_uint2(0u, 0u) : c;
      }
#pragma unroll
      for (int i = 0; i < W; ++i) w[j][i] = nx[j][i];
    }
  }
}

// Rows of more than 16384 columns: a block per row, read once for the maximum and again (from cache) for the codes.
template <typename T>
__global__ void __launch_bounds__(QI_MAX_THREADS) k_quantize_long_i8(const T* __restrict__ X, int K, int64_t ldx,
                                                                     const float* __restrict__ inv_s,
                                                                     int8_t* __restrict__ Xq, float* __restrict__ sx) {
  __shared__ uint32_t part[QI_MAX_THREADS / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t m = blockIdx.x;
  const T* row = X + m * ldx;
  const int nv = K >> 3, lane = threadIdx.x & 31;
  const auto fetch = [&](int v, float(&f)[8], float(&s)[8]) {
    uint32_t w[Elem<T>::kWords];
    load8(row + 8 * v, w);
    Elem<T>::unpack(w, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = inv_s ? __ldg(inv_s + 8 * v + i) : 1.0f;
  };
  uint32_t a = 0u;
#pragma unroll 4
  for (int v = threadIdx.x; v < nv; v += QI_MAX_THREADS) {
    float f[8], s[8];
    fetch(v, f, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) a = umax(a, abs_bits(__fmul_rn(f[i], s[i])));
  }
  a = __reduce_max_sync(0xFFFFFFFFu, a);
  if (lane == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
  a = __reduce_max_sync(0xFFFFFFFFu, part[lane & (QI_MAX_THREADS / 32 - 1)]);
  float scale, mul;
  i8_scale(a, scale, mul);
  if (threadIdx.x == 0) sx[m] = scale;
#pragma unroll 4
  for (int v = threadIdx.x; v < nv; v += QI_MAX_THREADS) {
    float f[8], s[8];
    fetch(v, f, s);
    const uint2 c = i8_codes(f, s, mul);
    *reinterpret_cast<uint2*>(Xq + m * K + 8 * v) = mul == 0.0f ? make_uint2(0u, 0u) : c;
  }
}

}  // namespace svdq
