// Channels-last group norm with an activation, and its form that quantizes for the int8 GEMM.
//   y = act((x - mean_g) rstd_g gamma_c + beta_c),  rstd = 1 / sqrt(var + eps), statistics over the S rows of a
//   sample and the C / G channels of a group
//
// Bound by memory: x read, y written, 4 bytes an element for 16-bit types.  Every output needs every input of
// its group, so there are two passes over the rows, in one of two forms:
//   k_group_norm   one launch; the blocks of a sample (up to eight, a cluster) keep its rows in shared memory between
//                  the passes and merge their statistics there: x is read once.  For samples that fit.
//   k_group_stats, k_group_apply   two launches over the same blocks of rows, the second a programmatic dependent of
//                  the first and walking its rows backwards (the rows read last are the ones L2 still has).
//                  Each block of the first leaves (mean, M2) of its rows per group, each block of the second
//                  merges those of its sample: nothing needs clearing, no block waits for another.
// The order of every sum is fixed.
// Measured: a megapixel of 128 bf16 channels with SiLU 139 us, 0.83 of the copy bandwidth (0.8 GB, 64 MB of it
// from L2); 2 x 4096 x 640 11.2 us (9.7 without SiLU; two launches' latencies are 6 of it); 64 x 320 6.7 us (one
// launch).  Codes: 2 x 1024 x 1280 10.6 us, 16384 x 320 15.6 us (issue-bound: of a row's 64 threads 40 hold a vector).
//
// Statistics: a thread owns 8 consecutive channels (a 16-byte vector of a 16-bit type) of every rp-th row,
// whichever groups they fall in, and sums x - p and its square per channel, p the median of three of the
// group's values in the block: p lies among them, so the squares do not cancel however far the mean is from zero or
// one value, channel or row from the others.  Blocks are merged by n, mean and M2 = sum (x - mean)^2 (T. F. Chan, G.
// H. Golub and R. J. LeVeque, "Updating formulae and a pairwise algorithm for computing sample variances", 1979).
#pragma once
#include "gelu.cuh"
#include "int8.cuh"
#include "tc_i8.cuh"

namespace svdq {

enum : int { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU = 2 };

// Threads a block: 640 for large tensors, whose passes are bound by what is in flight (a megapixel of 128 channels: 139
// us, 8 % more with 512), 512 for small ones, whose folds and merges are shorter with fewer rows at a time (64 rows
// of 320: 6.7 us, 7.1 with 640), and where codes are made (their registers).
constexpr int GN_MAX_THREADS = 640;
constexpr int GN_SMALL_THREADS = 512;
constexpr int GN_MAX_C = 8 * GN_SMALL_THREADS;
// Rows a thread takes at a time (and as many on their way): 64 bytes of them; two where codes are made, whose values
// wait in registers for their row's maximum (2 x 1024 x 1280: 10.2 us, 11.3 with four).
template <typename T, bool QUANT>
constexpr int GN_UNROLL = QUANT ? 2 : 8 / (int)sizeof(T);

struct GroupNormArgs {
  const void* X;
  int64_t ldx;
  int S, C, G;
  int nv;                 // 8-channel vectors a row, the last one possibly short
  int rp1;                // first pass: nv threads a row, rp1 rows at a time
  int l2, rp2;            // second pass: l2 threads a row (nv, or for codes whole warps or a power of two), rp2 rows
  int P;                  // blocks a sample, of `rows` rows each, the last one what is left
  int rows;
  float2* part;           // [sample][P][G]: (mean, M2) of a block's rows
  const float* gamma;
  const float* beta;
  float eps;
  int act;
  int hot;                // rows of a block before those that L2 is to hold until the second pass
  int streaming;          // Y is larger than L2 would keep: stores that do not displace X
  void* Y;
  int64_t ldy;
  const float* inv_s;
  int8_t* Xq;
  float* sx;
};

// Eight float32 parameters of channels c.. (c + 8 <= C where VEC).
template <bool VEC>
SVDQ_DEV void gn_params(const float* p, float other, int c, int C, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    float4 v = make_float4(other, other, other, other);
    if (p) {
      if constexpr (VEC) v = __ldg(reinterpret_cast<const float4*>(p + c + i));
      else v = make_float4(__ldg(p + min(c + i, C - 1)), __ldg(p + min(c + i + 1, C - 1)),
                           __ldg(p + min(c + i + 2, C - 1)), __ldg(p + min(c + i + 3, C - 1)));
    }
    f[i] = v.x;
    f[i + 1] = v.y;
    f[i + 2] = v.z;
    f[i + 3] = v.w;
  }
}

// Eight channels from c of the row at p.  VEC, every row on 16 bytes: as vectors.  Else from the aligned 16-byte pieces
// that hold them, shifted into place (2 x 4096 x 637 in one
// group: 18 us, 34 with loads and stores by the element); of a piece at least
// one byte is the row's, so that no other piece is touched, and what lies past the row's end is never used.  Plain
// loads: Y may be X.
template <typename T, bool VEC>
SVDQ_DEV void gn_load(const T* p, int c, int C, uint32_t (&w)[Elem<T>::kWords]) {
  constexpr int W = Elem<T>::kWords;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p + c)[i];
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  } else {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p + c), end = reinterpret_cast<uintptr_t>(p + C);
    const uint32_t off = (uint32_t)at & 15u;
    const uint4* piece = reinterpret_cast<const uint4*>(at - off);
    uint32_t q[W + 4];
#pragma unroll
    for (int i = 0; i <= W / 4; ++i) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (reinterpret_cast<uintptr_t>(piece + i) < end && (i < W / 4 || off)) v = piece[i];
      q[4 * i] = v.x;
      q[4 * i + 1] = v.y;
      q[4 * i + 2] = v.z;
      q[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < W + 2; ++i) q[i] = off & 8u ? q[i + 2] : q[i];
#pragma unroll
    for (int i = 0; i < W + 1; ++i) q[i] = off & 4u ? q[i + 1] : q[i];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = off & 2u ? __byte_perm(q[i], q[i + 1], 0x5432) : q[i];
  }
}

// Eight channels at p, wherever it lies: the widest stores its alignment allows (the same for all of a row's threads).
template <typename T>
SVDQ_DEV void gn_store_any(T* p, const uint32_t (&w)[Elem<T>::kWords]) {
  constexpr int W = Elem<T>::kWords;
  const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(p) & 15u;
  if ((off & 7u) == 0u) {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) reinterpret_cast<uint2*>(p)[i] = make_uint2(w[2 * i], w[2 * i + 1]);
  } else if ((off & 3u) == 0u) {
#pragma unroll
    for (int i = 0; i < W; ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
  } else {                                               // a 16-bit type on an odd element
    uint16_t* h = reinterpret_cast<uint16_t*>(p);
    h[0] = (uint16_t)w[0];
#pragma unroll
    for (int i = 0; i + 1 < W; ++i) *reinterpret_cast<uint32_t*>(h + 1 + 2 * i) = __byte_perm(w[i], w[i + 1], 0x5432);
    h[2 * W - 1] = (uint16_t)(w[W - 1] >> 16);
  }
}

// The same as vectors, and how L2 ranks the lines that the load brings: those to be read again soon before the rest.
SVDQ_DEV uint64_t l2_policy(bool again) {
  uint64_t first, normal;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
  asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
  return again ? normal : first;
}
template <typename T>
SVDQ_DEV void gn_load(const T* p, int c, uint64_t policy, uint32_t (&w)[Elem<T>::kWords]) {
#pragma unroll
  for (int i = 0; i < Elem<T>::kWords / 4; ++i)
    asm volatile("ld.global.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                 : "l"(reinterpret_cast<const uint4*>(p + c) + i), "l"(policy));
}

// M2 is never negative but for rounding; a NaN stays one.
SVDQ_DEV float gn_m2(float v) { return v < 0.0f ? 0.0f : v; }

// The pivot of the group of channels first.. in rows lo..hi: the median of its first channel in the first row, its
// middle one in the middle row and its last one in the last row.
template <typename T>
SVDQ_DEV float gn_pivot(const GroupNormArgs& a, const T* X, int lo, int hi, int first, int cg) {
  const float p = Elem<T>::to_f32(X[(int64_t)lo * a.ldx + first]);
  const float q = Elem<T>::to_f32(X[(int64_t)((lo + hi) >> 1) * a.ldx + first + (cg >> 1)]);
  const float r = Elem<T>::to_f32(X[(int64_t)(hi - 1) * a.ldx + first + cg - 1]);
  return fmaxf(fminf(p, q), fminf(fmaxf(p, q), r));
}

// (mean, M2) of each group from the n row slots' sums about the pivots, LANES lanes a group.
template <typename T, int LANES>
SVDQ_DEV void gn_group_sums(const GroupNormArgs& a, const T* X, int lo, int hi, int n, const float* sum, const float* sq,
                            float2* out) {
  constexpr int kGroups = 32 / LANES;                    // a warp's groups at a time
  const int width = 8 * a.nv, cg = a.C / a.G, lane = threadIdx.x & 31;
  const float count = (float)(hi - lo) * (float)cg, inv = 1.0f / count;
  for (int g0 = kGroups * (threadIdx.x >> 5); g0 < a.G; g0 += kGroups * (blockDim.x >> 5)) {   // uniform over a warp
    const int g = min(g0 + lane / LANES, a.G - 1);
    const float pivot = gn_pivot(a, X, lo, hi, g * cg, cg);
    float s1 = 0.0f, q1 = 0.0f;
#pragma unroll 4                                         // 64 loads in flight (2 x 1024 x 1280: 9.0 us, 9.6 without)
    for (int i = g * cg + lane % LANES; i < (g + 1) * cg; i += LANES) {
      float s[8], q[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s[k] = k < n ? sum[i + k * width] : 0.0f;
        q[k] = k < n ? sq[i + k * width] : 0.0f;
      }
      s1 += ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
      q1 += ((q[0] + q[1]) + (q[2] + q[3])) + ((q[4] + q[5]) + (q[6] + q[7]));
    }
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) {
      s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, o);
      q1 += __shfl_xor_sync(0xFFFFFFFFu, q1, o);
    }
    if (lane % LANES == 0 && g0 + lane / LANES < a.G) {
      const float d = s1 * inv;
      out[g] = make_float2(pivot + d, gn_m2(q1 - d * s1));
    }
  }
}

// First pass over the block's rows lo..hi: (mean, M2) of each group to out (shared or global memory).  sum and
// sq: 8 floats a thread each.  KEEP: the rows also go to `kept` (row by row, nv vectors).  LARGE: the tensor is larger
// than L2; the rows before a.hot are not to displace those after it, which the second pass reads first.
template <typename T, bool VEC, bool KEEP, bool LARGE>
SVDQ_DEV void gn_block_stats(const GroupNormArgs& a, const T* X, int lo, int hi, float* sum, float* sq, uint4* kept,
                             float2* out) {
  constexpr int W = Elem<T>::kWords, U = GN_UNROLL<T, false>;
  const int slot = threadIdx.x / a.nv, v = threadIdx.x - slot * a.nv, c = 8 * v;
  const int width = 8 * a.nv, cg = a.C / a.G;
  uint32_t x[U][W], nx[U][W];
  const uint64_t once = l2_policy(false), again = l2_policy(true);
  const auto fetch = [&](int r0, uint32_t(&x)[U][W]) {
    const uint64_t policy = r0 >= lo + a.hot ? again : once;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (r0 + u * a.rp1 >= hi) continue;
      const T* row = X + (int64_t)(r0 + u * a.rp1) * a.ldx;
      if constexpr (LARGE) gn_load<T>(row, c, policy, x[u]);
      else gn_load<T, VEC>(row, c, a.C, x[u]);
    }
  };
  // A thread a group finds the pivots, its loads in flight together with the rows', and hands them round in `sum` (each
  // thread for its channels: 24 loads, 0.6 us more).
  float own = 0.0f;
  if (threadIdx.x < a.G) own = gn_pivot(a, X, lo, hi, threadIdx.x * cg, cg);
  if (slot < a.rp1) fetch(lo + slot, x);
  if (threadIdx.x < a.G) sum[threadIdx.x] = own;
  for (int g = threadIdx.x + blockDim.x; g < a.G; g += blockDim.x) sum[g] = gn_pivot(a, X, lo, hi, g * cg, cg);
  __syncthreads();
  float pivot[8], s[8], q[8];
  if (slot < a.rp1) {
    int g = c / cg, left = cg * (g + 1) - c;             // the vector's channels, group by group
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool next = left == 0 && c + i < a.C;
      g += next ? 1 : 0;
      left = (next ? cg : left) - 1;
      pivot[i] = sum[g];
      s[i] = q[i] = 0.0f;
    }
  }
  __syncthreads();
  if (slot < a.rp1) {
    for (int r0 = lo + slot; r0 < hi; r0 += U * a.rp1) {
      fetch(r0 + U * a.rp1, nx);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * a.rp1;
        if (r >= hi) continue;
        float f[8];
        Elem<T>::unpack(x[u], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float e = f[i] - pivot[i];
          s[i] += e;
          q[i] = fmaf(e, e, q[i]);
        }
        if (KEEP) {
          uint4* k = kept + ((r - lo) * a.nv + v) * (W / 4);
#pragma unroll
          for (int i = 0; i < W / 4; ++i) k[i] = make_uint4(x[u][4 * i], x[u][4 * i + 1], x[u][4 * i + 2], x[u][4 * i + 3]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < W; ++i) x[u][i] = nx[u][i];
    }
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      *reinterpret_cast<float4*>(sum + slot * width + c + i) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
      *reinterpret_cast<float4*>(sq + slot * width + c + i) = make_float4(q[i], q[i + 1], q[i + 2], q[i + 3]);
    }
  }
  // row slots folded in half while there are many
  int n = a.rp1;
  for (; n > 8;) {
    const int h = (n + 1) >> 1;
    __syncthreads();
    for (int i = threadIdx.x; i < (n - h) * width; i += blockDim.x) {
      sum[i] += sum[i + h * width];
      sq[i] += sq[i + h * width];
    }
    n = h;
  }
  __syncthreads();
  // each group's channels and slots: by eight lanes, or a warp where few groups have many channels (2 x 4096 x 640 in
  // one group: 10.4 us, 13.1 with eight lanes)
  if (a.G <= 4) gn_group_sums<T, 32>(a, X, lo, hi, n, sum, sq, out);
  else gn_group_sums<T, 8>(a, X, lo, hi, n, sum, sq, out);
}

// Running merge of blocks' (n, mean, M2) against a common base: n, sum n (mean - base), sum n (mean - base)^2, M2.
struct GnMerge {
  float n = 0.0f, m = 0.0f, e2 = 0.0f, m2 = 0.0f;
  SVDQ_DEV void add(float2 v, float base, float k) {
    const float e = v.x - base;
    n += k;
    m = fmaf(k, e, m);
    e2 = fmaf(k * e, e, e2);
    m2 += v.y;
  }
  // mean and 1 / sqrt(var + eps)
  SVDQ_DEV float2 result(float base, float eps) const {
    const float d = m / n;
    return make_float2(base + d, __frsqrt_rn((m2 + gn_m2(e2 - d * m)) / n + eps));
  }
};

// y / (1 + exp(-y)), two elements sharing a reciprocal, 1 / d0 = d1 / (d0 d1): three special-function operations a
// pair instead of four, which bound the pass (16 a cycle and SM).  exp(-y) is cut at y = -40, where the result is
// below 2e-16 in magnitude either way, so that the product of two d stays in range.
SVDQ_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
SVDQ_DEV float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
SVDQ_DEV float2 silu_f32x2(float2 y) {
  const float2 z = mul_f32x2(f2(-1.44269504f), make_float2(fmaxf(y.x, -40.0f), fmaxf(y.y, -40.0f)));
  const float2 d = add_f32x2(make_float2(ex2(z.x), ex2(z.y)), f2(1.0f));
  const float r = rcp(d.x * d.y);
  return mul_f32x2(y, mul_f32x2(f2(r), make_float2(d.y, d.x)));
}

template <int ACT>
SVDQ_DEV float2 gn_act(float2 y) {
  if constexpr (ACT == ACT_SILU) return silu_f32x2(y);
  else if constexpr (ACT == ACT_GELU) return gelu_f32x2(y);
  else return y;
}

// A thread's part of the second pass, set up before the statistics are there: its place (l2 threads a row), the
// parameters of its channels, and its first rows (not where they are in shared memory).
template <typename T, bool VEC, bool QUANT, bool KEEP>
struct GnApply {
  static constexpr int W = Elem<T>::kWords, U = GN_UNROLL<T, QUANT>;
  int slot, v, c;
  bool on;
  float ga[8], be[8], is[QUANT ? 8 : 1];
  uint32_t x[U][W], nx[U][W];

  SVDQ_DEV GnApply(const GroupNormArgs& a) {
    slot = threadIdx.x / a.l2;
    v = threadIdx.x - slot * a.l2;
    c = 8 * v;
    on = slot < a.rp2 && v < a.nv;
    if (on) {
      gn_params<VEC>(a.gamma, 1.0f, c, a.C, ga);
      gn_params<VEC>(a.beta, 0.0f, c, a.C, be);
      if constexpr (QUANT) gn_params<VEC>(a.inv_s, 1.0f, c, a.C, is);
    }
  }
  // Rows r0 - slot, r0 - slot - rp2, ... down to lo; at: the first of them in X.
  SVDQ_DEV void fetch(const GroupNormArgs& a, const T* at, const uint4* kept, int lo, int r0, uint32_t (&x)[U][W]) {
    if (!on) return;
    const int64_t step = a.rp2 * a.ldx;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 - u * a.rp2 - slot;
      if (r < lo) continue;
      if constexpr (KEEP) {
        const uint4* k = kept + ((r - lo) * a.nv + v) * (W / 4);
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
          const uint4 d = k[i];
          x[u][4 * i] = d.x;
          x[u][4 * i + 1] = d.y;
          x[u][4 * i + 2] = d.z;
          x[u][4 * i + 3] = d.w;
        }
      } else {
        gn_load<T, VEC>(at - u * step, c, a.C, x[u]);
      }
    }
  }
};

// Second pass over rows lo..hi of sample b, from the last to the first (t.fetch has the first step's rows).  stat:
// (mean, rstd) of the groups; KEEP: the rows are in `kept`.  QUANT: instead of Y, rows of 8-bit codes and their
// scales.  A row's l2 threads are whole warps, or 4 to 32 lanes of one, a power of two: its maximum is a reduction
// over lanes, and over warps through `top` (two buffers of U words a warp; one barrier of the row's warps a step: l2
// >= 64 there, so at most 8 rows and barriers).
template <typename T, bool VEC, bool QUANT, bool KEEP, int ACT>
SVDQ_DEV void gn_apply_loop(const GroupNormArgs& a, GnApply<T, VEC, QUANT, KEEP>& t, const T* X, int b, int lo, int hi,
                            const float2 (&mu)[4], const float2 (&ga)[4], const float2 (&be)[4], const uint4* kept,
                            uint32_t* top) {
  constexpr int W = Elem<T>::kWords, U = GN_UNROLL<T, QUANT>;
  const int slot = t.slot, v = t.v, c = t.c, lane = threadIdx.x & 31;
  const bool on = t.on;
  const auto value = [&](const uint32_t(&w)[W], float2(&y)[4]) {
    float f[8];
    Elem<T>::unpack(w, f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      y[i] = gn_act<ACT>(fma_f32x2(sub_f32x2(make_float2(f[2 * i], f[2 * i + 1]), mu[i]), ga[i], be[i]));
  };
  const int64_t istep = a.rp2 * a.ldx, ostep = a.rp2 * a.ldy;
  const T* in = X + (hi - 1 - slot) * a.ldx;
  T* out = QUANT ? nullptr : static_cast<T*>(a.Y) + ((int64_t)b * a.S + hi - 1 - slot) * a.ldy + c;
  const int nw = a.l2 >> 5;                              // warps a row, 0: part of one
  int buf = 0;
  for (int r0 = hi - 1; r0 >= lo; r0 -= U * a.rp2) {     // uniform over the block
    in -= U * istep;
    if (!KEEP) t.fetch(a, in, kept, lo, r0 - U * a.rp2, t.nx);
    if constexpr (!QUANT) {
      if (on) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = r0 - u * a.rp2 - slot;
          if (r < lo) continue;
          float2 y[4];
          value(t.x[u], y);
          const float f[8] = {y[0].x, y[0].y, y[1].x, y[1].y, y[2].x, y[2].y, y[3].x, y[3].y};
          T* p = out - u * ostep;
          if constexpr (VEC) {
            uint32_t o[W];
            Elem<T>::pack(f, o);
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
              const uint4 d = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
              if (a.streaming) __stcs(reinterpret_cast<uint4*>(p) + i, d);
              else reinterpret_cast<uint4*>(p)[i] = d;
            }
          } else if (c + 8 <= a.C) {
            uint32_t o[W];
            Elem<T>::pack(f, o);
            gn_store_any<T>(p, o);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c + i < a.C) p[i] = Elem<T>::from_f32(f[i]);
          }
        }
      }
      out -= U * ostep;
    } else {
      float2 y[U][4];
      uint32_t m[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float top_u = 0.0f;
        if (on && r0 - u * a.rp2 - slot >= lo) {
          value(t.x[u], y[u]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[u][i] = mul_f32x2(y[u][i], make_float2(t.is[2 * i], t.is[2 * i + 1]));
            top_u = max_abs(top_u, y[u][i].x, y[u][i].y);            // C % 16 == 0: whole vectors
          }
        }
        m[u] = __float_as_uint(top_u);
      }
      __syncwarp();                                      // the lanes parted above
      if (nw) {
#pragma unroll
        for (int u = 0; u < U; ++u) m[u] = __reduce_max_sync(0xFFFFFFFFu, m[u]);
      } else {
        for (int o = a.l2 >> 1; o; o >>= 1)
#pragma unroll
          for (int u = 0; u < U; ++u) m[u] = umax(m[u], __shfl_xor_sync(0xFFFFFFFFu, m[u], o));
      }
      if (nw > 1) {
        uint32_t* now = top + buf * U * (blockDim.x >> 5);           // [u][warp]
        const int warp = threadIdx.x >> 5;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (lane == u) now[u * (blockDim.x >> 5) + warp] = m[u];
        // Only the warps of this row wait for one another, so that the rows' chains of latencies overlap (a row's
        // threads are whole warps; warps past the last row take no part).
        if (slot < a.rp2) {
          asm volatile("bar.sync %0, %1;" ::"r"(1 + slot), "r"(a.l2) : "memory");
#pragma unroll
          for (int u = 0; u < U; ++u)
            for (int k = 0; k < nw; ++k) m[u] = umax(m[u], now[u * (blockDim.x >> 5) + slot * nw + k]);
        }
        buf ^= 1;
      }
      // Of a row's first 2 U threads, j works out the multiplier of its row j of the U or, from U on, the scale of row
      // j - U: one division for all.
      static_assert((U & (U - 1)) == 0 && 2 * U <= 4, "at least 2 U lanes a row");
      const int group = min(a.l2, 32), j = lane & (group - 1) & (U - 1);
      uint32_t own = m[0];
#pragma unroll
      for (int u = 1; u < U; ++u) own = j == u ? m[u] : own;
      const float either = i8_scale_or_mul(own, (lane & U) != 0);
      if (v >= U && v < 2 * U && slot < a.rp2 && r0 - j * a.rp2 - slot >= lo)
        a.sx[(int64_t)b * a.S + r0 - j * a.rp2 - slot] = either;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 - u * a.rp2 - slot;
        const float mul_u = __shfl_sync(0xFFFFFFFFu, either, u, group);
        if (on && r >= lo) {
          const uint2 code = i8_codes(y[u], mul_u);
          *reinterpret_cast<uint2*>(a.Xq + ((int64_t)b * a.S + r) * a.C + c) = mul_u == 0.0f ? make_uint2(0u, 0u) : code;
        }
      }
    }
    if (KEEP) {
      t.fetch(a, nullptr, kept, lo, r0 - U * a.rp2, t.x);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < W; ++i) t.x[u][i] = t.nx[u][i];
    }
  }
}

template <typename T, bool VEC, bool QUANT, bool KEEP>
SVDQ_DEV void gn_apply_rows(const GroupNormArgs& a, GnApply<T, VEC, QUANT, KEEP>& t, const T* X, int b, int lo, int hi,
                            const float2* stat, const uint4* kept, uint32_t* top) {
  const int c = t.c, cg = a.C / a.G;
  float2 mu[4], ga[4], be[4];
  if (t.on) {
    int g = c / cg, left = cg * (g + 1) - c;             // the vector's channels, group by group
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool next = left == 0 && c + i < a.C;
      g += next ? 1 : 0;
      left = (next ? cg : left) - 1;
      const float2 st = stat[g];
      m[i] = st.x;
      t.ga[i] *= st.y;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mu[i] = make_float2(m[2 * i], m[2 * i + 1]);
      ga[i] = make_float2(t.ga[2 * i], t.ga[2 * i + 1]);
      be[i] = make_float2(t.be[2 * i], t.be[2 * i + 1]);
    }
  }
  if (a.act == ACT_NONE) gn_apply_loop<T, VEC, QUANT, KEEP, ACT_NONE>(a, t, X, b, lo, hi, mu, ga, be, kept, top);
  else if (a.act == ACT_SILU) gn_apply_loop<T, VEC, QUANT, KEEP, ACT_SILU>(a, t, X, b, lo, hi, mu, ga, be, kept, top);
  else gn_apply_loop<T, VEC, QUANT, KEEP, ACT_GELU>(a, t, X, b, lo, hi, mu, ga, be, kept, top);
}

template <typename T, bool VEC, bool LARGE>
__global__ void __launch_bounds__(GN_MAX_THREADS, 1) k_group_stats(const GroupNormArgs a) {
  __shared__ __align__(16) float sum[8 * GN_MAX_THREADS], sq[8 * GN_MAX_THREADS];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x / a.P, p = blockIdx.x - b * a.P;
  const int lo = p * a.rows, hi = min(a.S, lo + a.rows);
  gn_block_stats<T, VEC, false, LARGE>(a, static_cast<const T*>(a.X) + (int64_t)b * a.S * a.ldx, lo, hi, sum, sq, nullptr,
                                a.part + (int64_t)blockIdx.x * a.G);
}

// The sample's P partials of each group are merged by strips of threads: thread (j, g) takes every J-th block, ten
// loads in flight, and the strips are joined through shared memory.
constexpr int GN_MERGE_LOADS = 10;
template <typename T, bool VEC, bool QUANT>
__global__ void __launch_bounds__(QUANT ? GN_SMALL_THREADS : GN_MAX_THREADS, 1) k_group_apply(const GroupNormArgs a) {
  extern __shared__ __align__(16) float2 stat[];         // G of (mean, rstd), then a GnMerge a thread
  __shared__ uint32_t top[2 * GN_UNROLL<T, QUANT> * GN_MAX_THREADS / 32];
  const int b = blockIdx.x / a.P, p = blockIdx.x - b * a.P;
  const int lo = p * a.rows, hi = min(a.S, lo + a.rows);
  const float cg = (float)(a.C / a.G);
  GnMerge* strip = reinterpret_cast<GnMerge*>(stat + (a.G + 1) / 2 * 2);
  const T* X = static_cast<const T*>(a.X) + (int64_t)b * a.S * a.ldx;
  // Inputs may be read before the wait: the first pass started after everything before it was done.
  GnApply<T, VEC, QUANT, false> t(a);
  t.fetch(a, X + (hi - 1 - t.slot) * a.ldx, nullptr, lo, hi - 1, t.x);
  griddep_wait();
  griddep_launch_dependents();
  const float2* part = a.part + (int64_t)b * a.P * a.G;
  const int J = max(1, (int)blockDim.x / a.G), j = threadIdx.x / a.G, last_rows = a.S - (a.P - 1) * a.rows;
  for (int g0 = 0; g0 < a.G; g0 += blockDim.x) {         // one round unless there are more groups than threads
    const int g = g0 + (J > 1 ? threadIdx.x - j * a.G : threadIdx.x);
    GnMerge acc;
    if ((J > 1 ? j < J : true) && g < a.G) {
      const float base = part[g].x;
      for (int p0 = J > 1 ? j : 0; p0 < a.P; p0 += GN_MERGE_LOADS * J) {
        float2 v[GN_MERGE_LOADS];
#pragma unroll
        for (int k = 0; k < GN_MERGE_LOADS; ++k)
          if (p0 + k * J < a.P) v[k] = part[(int64_t)(p0 + k * J) * a.G + g];
#pragma unroll
        for (int k = 0; k < GN_MERGE_LOADS; ++k)
          if (p0 + k * J < a.P) acc.add(v[k], base, cg * (float)(p0 + k * J == a.P - 1 ? last_rows : a.rows));
      }
      if (J == 1) stat[g] = acc.result(base, a.eps);
      else strip[j * a.G + g] = acc;
    }
  }
  if (J > 1) {
    int n = J;
    for (; n > 8;) {
      const int h = (n + 1) >> 1;
      __syncthreads();
      for (int i = threadIdx.x; i < (n - h) * a.G; i += blockDim.x) {
        strip[i].n += strip[i + h * a.G].n;
        strip[i].m += strip[i + h * a.G].m;
        strip[i].e2 += strip[i + h * a.G].e2;
        strip[i].m2 += strip[i + h * a.G].m2;
      }
      n = h;
    }
    __syncthreads();
    if (threadIdx.x < a.G) {
      GnMerge acc = strip[threadIdx.x];
#pragma unroll
      for (int k = 1; k < 8; ++k)
        if (k < n) {
          const GnMerge o = strip[k * a.G + threadIdx.x];
          acc.n += o.n;
          acc.m += o.m;
          acc.e2 += o.e2;
          acc.m2 += o.m2;
        }
      stat[threadIdx.x] = acc.result(part[threadIdx.x].x, a.eps);
    }
  }
  __syncthreads();
  gn_apply_rows<T, VEC, QUANT, false>(a, t, X, b, lo, hi, stat, nullptr, top);
}

// Floats of k_group_norm's shared memory before the kept rows: own partials and statistics of G groups, sums and
// squares of 8 values a thread (a multiple of 4).
__host__ __device__ constexpr int gn_fixed_floats(int G, int threads) { return (4 * G + 16 * threads + 3) / 4 * 4; }

template <typename T, bool VEC, bool QUANT>
__global__ void __launch_bounds__(GN_SMALL_THREADS, 1) k_group_norm(const GroupNormArgs a) {
  extern __shared__ __align__(16) float gn_smem[];
  __shared__ uint32_t top[2 * GN_UNROLL<T, QUANT> * GN_MAX_THREADS / 32];
  float* sum = gn_smem;
  float* sq = sum + 8 * blockDim.x;
  float2* mine = reinterpret_cast<float2*>(sq + 8 * blockDim.x);
  float2* stat = mine + a.G;
  uint4* kept = reinterpret_cast<uint4*>(gn_smem + gn_fixed_floats(a.G, blockDim.x));
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x / a.P, p = blockIdx.x - b * a.P;
  const int lo = p * a.rows, hi = min(a.S, lo + a.rows);
  const T* X = static_cast<const T*>(a.X) + (int64_t)b * a.S * a.ldx;
  gn_block_stats<T, VEC, true, false>(a, X, lo, hi, sum, sq, kept, mine);
  GnApply<T, VEC, QUANT, true> t(a);                     // its loads on their way while the blocks meet
  __syncwarp();
  if (a.P > 1) cluster_sync_all();
  else __syncthreads();
  const float cg = (float)(a.C / a.G);
  for (int g = threadIdx.x; g < a.G; g += blockDim.x) {
    float2 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < a.P) v[k] = a.P > 1 ? ld_cluster_f2(map_to_rank(smem_u32(mine + g), (uint32_t)k)) : mine[g];
    GnMerge acc;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < a.P) acc.add(v[k], v[0].x, cg * (float)min(a.rows, a.S - k * a.rows));
    stat[g] = acc.result(v[0].x, a.eps);
  }
  __syncwarp();
  if (a.P > 1) cluster_sync_all();                       // no block leaves while another reads its partials
  else __syncthreads();
  t.fetch(a, X, kept, lo, hi - 1, t.x);
  gn_apply_rows<T, VEC, QUANT, true>(a, t, X, b, lo, hi, stat, kept, top);
}

}  // namespace svdq
