// Channels-last group norm with an activation, and its form that quantizes for the int8 GEMM.
//   y = act((x - mean_g) rstd_g gamma_c + beta_c),  statistics over the S rows and C / G channels of a group
#pragma once
#include "gelu.cuh"
#include "int8.cuh"

namespace svdq {

enum : int { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU = 2 };

SVDQ_DEV float apply_act(float y, int act) {
  if (act == ACT_SILU) return __fdividef(y, 1.0f + __expf(-y));
  if (act == ACT_GELU) return gelu_f32(y);
  return y;
}

// Statistics of one (sample, group): a block, two passes; stats[b G + g] = {mean, 1 / sqrt(var + eps)}.
template <typename T>
__global__ void __launch_bounds__(256) k_group_stats(const T* __restrict__ X, int64_t S, int C, int64_t ldx, int G,
                                                     float eps, float2* __restrict__ stats) {
  __shared__ float red[8];
  griddep_wait();
  const int cg = C / G;
  const T* base = X + (int64_t)(blockIdx.x / G) * S * ldx + (int64_t)(blockIdx.x % G) * cg;
  const int64_t n = S * cg;
  float total[2];
  for (int pass = 0; pass < 2; ++pass) {
    float s = 0.0f;
    for (int64_t i = threadIdx.x; i < n; i += 256) {
      const float x = Elem<T>::to_f32(base[i / cg * ldx + i % cg]);
      s += pass == 0 ? x : (x - total[0]) * (x - total[0]);
    }
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0f;
    for (int i = 0; i < 8; ++i) s += red[i];
    total[pass] = s / (float)n;
  }
  if (threadIdx.x == 0) stats[blockIdx.x] = make_float2(total[0], 1.0f / sqrtf(total[1] + eps));
}

template <typename T, bool QUANT>
__global__ void __launch_bounds__(256) k_group_apply(const T* __restrict__ X, int64_t S, int C, int64_t ldx, int G,
                                                     const float2* __restrict__ stats, const float* __restrict__ gamma,
                                                     const float* __restrict__ beta, int act, T* __restrict__ Y,
                                                     int64_t ldy, const float* __restrict__ inv_s,
                                                     int8_t* __restrict__ Xq, float* __restrict__ sx) {
  __shared__ uint32_t part[8];
  griddep_wait();
  const int64_t row = blockIdx.x, b = row / S;
  const int cg = C / G;
  auto value = [&](int c) {
    const float2 st = stats[b * G + c / cg];
    float y = __fmaf_rn((Elem<T>::to_f32(X[row * ldx + c]) - st.x) * st.y, gamma ? gamma[c] : 1.0f, beta ? beta[c] : 0.0f);
    return apply_act(y, act);
  };
  if constexpr (!QUANT) {
    for (int c = threadIdx.x; c < C; c += 256) Y[row * ldy + c] = Elem<T>::from_f32(value(c));
  } else {
    uint32_t a = 0u;
    for (int c = threadIdx.x; c < C; c += 256) a = umax(a, abs_bits(__fmul_rn(value(c), inv_s ? inv_s[c] : 1.0f)));
    a = __reduce_max_sync(0xFFFFFFFFu, a);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
    __syncthreads();
    for (int i = 0; i < 8; ++i) a = umax(a, part[i]);
    float scale, mul;
    i8_scale(a, scale, mul);
    if (threadIdx.x == 0) sx[row] = scale;
    for (int c = threadIdx.x; c < C; c += 256)
      Xq[row * C + c] = (int8_t)i8_code(__fmul_rn(value(c), inv_s ? inv_s[c] : 1.0f), mul);
  }
}

}  // namespace svdq
