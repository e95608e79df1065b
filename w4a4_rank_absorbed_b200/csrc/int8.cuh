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

// 16 consecutive bytes of a row hold Elem<T>::kVec elements; a vector of 8 elements is kRegs words.
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
// Code of x (0 whatever x is where mul = 0: an infinite x times 0 is NaN, which has no integer).
SVDQ_DEV int i8_code(float x, float mul) { return mul == 0.0f ? 0 : __float2int_rn(__fmul_rn(x, mul)); }
SVDQ_DEV uint32_t pack_i8x4(int a, int b, int c, int d) {
  return (uint32_t)(a & 0xFF) | ((uint32_t)(b & 0xFF) << 8) | ((uint32_t)(c & 0xFF) << 16) | ((uint32_t)(d & 0xFF) << 24);
}

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

// Activation quantization: one block per row, two passes over it (the second from cache).
template <typename T>
__global__ void __launch_bounds__(256) k_quantize_act_i8(const T* __restrict__ X, int K, int64_t ldx,
                                                         const float* __restrict__ inv_s, int8_t* __restrict__ Xq,
                                                         float* __restrict__ sx) {
  __shared__ uint32_t part[8];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t m = blockIdx.x;
  const T* row = X + m * ldx;
  const int nv = K >> 3;
  uint32_t a = 0u;
  for (int v = threadIdx.x; v < nv; v += 256) {
    uint32_t w[Elem<T>::kWords];
    float f[8];
    load8(row + 8 * v, w);
    Elem<T>::unpack(w, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) a = umax(a, abs_bits(inv_s ? __fmul_rn(f[i], __ldg(inv_s + 8 * v + i)) : f[i]));
  }
  a = __reduce_max_sync(0xFFFFFFFFu, a);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) a = umax(a, part[i]);
  float scale, mul;
  i8_scale(a, scale, mul);
  if (threadIdx.x == 0) sx[m] = scale;
  for (int v = threadIdx.x; v < nv; v += 256) {
    uint32_t w[Elem<T>::kWords];
    float f[8];
    int q[8];
    load8(row + 8 * v, w);
    Elem<T>::unpack(w, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = i8_code(inv_s ? __fmul_rn(f[i], __ldg(inv_s + 8 * v + i)) : f[i], mul);
    *reinterpret_cast<uint2*>(Xq + m * K + 8 * v) =
        make_uint2(pack_i8x4(q[0], q[1], q[2], q[3]), pack_i8x4(q[4], q[5], q[6], q[7]));
  }
}

}  // namespace svdq
