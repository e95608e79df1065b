// Int8 GEMM with scales per token and channel:
//   Y[m, n] = f32(f32(f32(acc) sx[m]) sw[n]) + bias[n],  acc = sum_k Xq[m, k] Wq[n, k]  (int32, exact for K < 2^17)
// rounded once to the type of Y.
#pragma once
#include "int8.cuh"

namespace svdq {

struct LinearI8Args {
  const float* sx;
  const float* sw;
  const float* bias;
  void* Y;
  int y_type;
  int64_t ldy;
  int M, N, K;
};

SVDQ_DEV float i8_dequant(int acc, float sx, float sw, float bias) {
  return __fmaf_rn(__fmul_rn(__int2float_rn(acc), sx), sw, bias);
}
SVDQ_DEV void store_y(void* Y, int type, int64_t at, float y) {
  if (type == DT_BF16) static_cast<__nv_bfloat16*>(Y)[at] = __float2bfloat16_rn(y);
  else if (type == DT_FP16) static_cast<__half*>(Y)[at] = __float2half_rn(y);
  else static_cast<float*>(Y)[at] = y;
}

// 64 x 64 outputs a block, 4 x 4 a thread, four products an instruction.
__global__ void __launch_bounds__(256) k_linear_i8(const int8_t* __restrict__ Xq, const int8_t* __restrict__ Wq,
                                                   const LinearI8Args a) {
  __shared__ uint32_t xs[64][17], ws[64][17];
  griddep_wait();
  const int m0 = blockIdx.x * 64, n0 = blockIdx.y * 64;
  const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += 64) {
    const int r = threadIdx.x / 4, c = (threadIdx.x % 4) * 16;
    const bool kin = k0 + c < a.K;
    const uint4 z = make_uint4(0, 0, 0, 0);
    const uint4 x = kin && m0 + r < a.M ? *reinterpret_cast<const uint4*>(Xq + (int64_t)(m0 + r) * a.K + k0 + c) : z;
    const uint4 w = kin && n0 + r < a.N ? *reinterpret_cast<const uint4*>(Wq + (int64_t)(n0 + r) * a.K + k0 + c) : z;
    const int j = c / 4;
    xs[r][j] = x.x; xs[r][j + 1] = x.y; xs[r][j + 2] = x.z; xs[r][j + 3] = x.w;
    ws[r][j] = w.x; ws[r][j + 1] = w.y; ws[r][j + 2] = w.z; ws[r][j + 3] = w.w;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int l = 0; l < 4; ++l) acc[i][l] = __dp4a((int)xs[tm * 4 + i][k], (int)ws[tn + 16 * l][k], acc[i][l]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int l = 0; l < 4; ++l) {
      const int m = m0 + tm * 4 + i, n = n0 + tn + 16 * l;
      if (m < a.M && n < a.N)
        store_y(a.Y, a.y_type, (int64_t)m * a.ldy + n,
                i8_dequant(acc[i][l], __ldg(a.sx + m), __ldg(a.sw + n), a.bias ? __ldg(a.bias + n) : 0.0f));
    }
}

}  // namespace svdq
