// Channels-last group norm with an activation, and its form that quantizes for the int8 GEMM.
//   y = act((x - mean_g) rstd_g gamma_c + beta_c),  rstd = 1 / sqrt(var + eps), statistics over the S rows of a
//   sample and the C / G channels of a group
//
// Bound by memory: x read, y written, 4 bytes an element for 16-bit types.  Every output needs every input of
// its group, so x is read twice, the second time from L2 as far as it holds it: two launches over the same
// rows, the second a programmatic dependent of the first and walking its rows backwards (the rows read last
// are the ones L2 still has).  Between them each block of the first leaves (mean, M2) of its rows per group,
// and each block of the second merges those of its sample: nothing needs clearing beforehand, no block
// waits for another, and the order of every sum is fixed.
//
// Statistics: a thread owns 8 consecutive channels (a 16-byte vector of a 16-bit type) of every rp-th row,
// whichever groups they fall in, and sums x - p and its square per channel, p the block's first row: p lies in
// the channel's own range, so the squares do not cancel however far the mean is from zero.  Channels, blocks and
// groups are then merged by n, mean and M2 = sum (x - mean)^2 (T. F. Chan, G. H. Golub and R. J. LeVeque, "Updating
// formulae and a pairwise algorithm for computing sample variances", 1979).
#pragma once
#include "gelu.cuh"
#include "int8.cuh"

namespace svdq {

enum : int { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU = 2 };

constexpr int GN_MAX_THREADS = 512;
constexpr int GN_MAX_C = 8 * GN_MAX_THREADS;
// Rows a thread has in flight: 128 bytes of them.
template <typename T>
constexpr int GN_UNROLL = 16 / (int)sizeof(T);
constexpr int GN_QROWS = 4;                    // rows a thread quantizes at a time

struct GroupNormArgs {
  const void* X;
  int64_t ldx;
  int S, C, G;
  int nv;                 // 8-channel vectors a row, the last one possibly short
  int rp;                 // rows a block takes at a time: threads / nv
  int P;                  // blocks a sample, of `rows` rows each, the last one what is left
  int rows;
  int parts;              // entries of part a sample: the first pass's blocks, or 1 once merged (of part_rows rows)
  int part_rows;
  float2* part;           // [sample][parts][G]: (mean, M2) of a block's rows
  const float* gamma;
  const float* beta;
  float eps;
  int act;
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

// Eight channels from c of the row at p: one vector where every row starts on 16 bytes (VEC), else one by one;
// channels past C are 0.  Plain loads: Y may be X.
template <typename T, bool VEC>
SVDQ_DEV void gn_load(const T* p, int c, int C, uint32_t (&w)[Elem<T>::kWords]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < Elem<T>::kWords / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p + c)[i];
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  } else {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < C ? Elem<T>::to_f32(p[c + i]) : 0.0f;
    Elem<T>::pack(f, w);
  }
}

// M2 is never negative but for rounding; a NaN stays one.
SVDQ_DEV float gn_m2(float v) { return v < 0.0f ? 0.0f : v; }
template <typename T, bool VEC>
__global__ void __launch_bounds__(GN_MAX_THREADS) k_group_stats(const GroupNormArgs a) {
  constexpr int W = Elem<T>::kWords, U = GN_UNROLL<T>;
  __shared__ float sum[GN_MAX_C], sq[GN_MAX_C];          // [row slot][8 nv]: at most 8 values a thread
  const int b = blockIdx.x / a.P, p = blockIdx.x % a.P;
  const int lo = p * a.rows, hi = min(a.S, lo + a.rows);
  const int slot = threadIdx.x / a.nv, v = threadIdx.x % a.nv, c = 8 * v;
  const int width = 8 * a.nv;
  const T* X = static_cast<const T*>(a.X) + (int64_t)b * a.S * a.ldx;
  griddep_wait();
  griddep_launch_dependents();
  float pivot[8], s[8], q[8];
  if (slot < a.rp) {
    uint32_t w[W];
    gn_load<T, VEC>(X + lo * a.ldx, c, a.C, w);
    Elem<T>::unpack(w, pivot);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = q[i] = 0.0f;
    const auto add = [&](const uint32_t(&d)[W]) {
      float f[8];
      Elem<T>::unpack(d, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e = f[i] - pivot[i];
        s[i] += e;
        q[i] = fmaf(e, e, q[i]);
      }
    };
    for (int r0 = lo + slot; r0 < hi; r0 += U * a.rp) {
      uint32_t x[U][W];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (r0 + u * a.rp < hi) gn_load<T, VEC>(X + (int64_t)(r0 + u * a.rp) * a.ldx, c, a.C, x[u]);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (r0 + u * a.rp < hi) add(x[u]);
    }
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      *reinterpret_cast<float4*>(sum + slot * width + c + i) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
      *reinterpret_cast<float4*>(sq + slot * width + c + i) = make_float4(q[i], q[i + 1], q[i + 2], q[i + 3]);
    }
  }
  // the row slots' sums: folded in half while there are many, then one channel a thread
  int n = a.rp;
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
  // mean (less the pivot) and M2 of each channel, in place
  const float rows = (float)(hi - lo), inv = 1.0f / rows;
  for (int i = threadIdx.x; i < width; i += blockDim.x) {
    float s1 = sum[i], q1 = sq[i];
    for (int k = 1; k < n; ++k) {
      s1 += sum[i + k * width];
      q1 += sq[i + k * width];
    }
    const float d = s1 * inv;
    sq[i] = gn_m2(q1 - d * s1);
    sum[i] = d;
  }
  __syncthreads();
  if (slot == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[c + i] += pivot[i];
  }
  __syncthreads();
  // and of each group: eight lanes each
  const int cg = a.C / a.G, lane = threadIdx.x & 7;
  const float icg = 1.0f / (float)cg;
  for (int g0 = 4 * (threadIdx.x >> 5); g0 < a.G; g0 += blockDim.x >> 3) {     // uniform over a warp
    const int g = min(g0 + ((threadIdx.x >> 3) & 3), a.G - 1);
    const float base = sum[g * cg];
    float m = 0.0f, m2 = 0.0f, e2 = 0.0f;
    for (int i = lane; i < cg; i += 8) {
      const float e = sum[g * cg + i] - base;
      m += e;
      e2 = fmaf(e, e, e2);
      m2 += sq[g * cg + i];
    }
#pragma unroll
    for (int o = 4; o; o >>= 1) {
      m += __shfl_xor_sync(0xFFFFFFFFu, m, o);
      e2 += __shfl_xor_sync(0xFFFFFFFFu, e2, o);
      m2 += __shfl_xor_sync(0xFFFFFFFFu, m2, o);
    }
    m *= icg;
    if (lane == 0 && g0 + ((threadIdx.x >> 3) & 3) < a.G)
      a.part[(int64_t)blockIdx.x * a.G + g] = make_float2(base + m, m2 + rows * gn_m2(e2 - (float)cg * m * m));
  }
}

// (mean, M2) of one group over the P blocks of its sample: `part` is block 0's entry, `lanes` lanes of a warp
// work together (a power of two, `lane` among them); a block has `rows` of the S rows, the last what is left.
SVDQ_DEV float2 gn_merge(const float2* part, int G, int P, int rows, int S, int cg, int lane, int lanes) {
  const float base = part[0].x;
  float n = 0.0f, m = 0.0f, m2 = 0.0f, e2 = 0.0f;
#pragma unroll 8
  for (int p = lane; p < P; p += lanes) {
    const float2 v = part[(int64_t)p * G];
    const float k = (float)min(rows, S - p * rows) * (float)cg;
    const float e = v.x - base;
    n += k;
    m = fmaf(k, e, m);
    e2 = fmaf(k * e, e, e2);
    m2 += v.y;
  }
  for (int o = lanes >> 1; o; o >>= 1) {
    n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    m += __shfl_xor_sync(0xFFFFFFFFu, m, o);
    e2 += __shfl_xor_sync(0xFFFFFFFFu, e2, o);
    m2 += __shfl_xor_sync(0xFFFFFFFFu, m2, o);
  }
  m /= n;
  return make_float2(base + m, (m2 + gn_m2(e2 - n * m * m)) / n);      // mean, variance
}

SVDQ_DEV void gn_act(float (&y)[8], int act) {
  if (act == ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fdividef(y[i], 1.0f + __expf(-y[i]));
  } else if (act == ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 g = gelu_f32x2(make_float2(y[i], y[i + 1]));
      y[i] = g.x;
      y[i + 1] = g.y;
    }
  }
}

// The second pass.  QUANT: instead of Y, rows of 8-bit codes and their scales; a row's maximum is taken over the
// lanes of a warp that hold it and joined through shared memory (integer maximum: any order), GN_QROWS rows a
// thread at a time with one barrier.
template <typename T, bool VEC, bool QUANT>
__global__ void __launch_bounds__(GN_MAX_THREADS) k_group_apply(const GroupNormArgs a) {
  constexpr int W = Elem<T>::kWords, U = QUANT ? GN_QROWS : GN_UNROLL<T>;
  extern __shared__ float2 stat[];                       // G of (mean, rstd); QUANT: then 3 x GN_QROWS rp row maxima
  const int b = blockIdx.x / a.P, p = blockIdx.x % a.P;
  const int lo = p * a.rows, hi = min(a.S, lo + a.rows);
  const int slot = threadIdx.x / a.nv, v = threadIdx.x % a.nv, c = 8 * v;
  const int cg = a.C / a.G, lane = threadIdx.x & 31;
  const bool work = slot < a.rp;
  uint32_t* top = reinterpret_cast<uint32_t*>(stat + a.G);
  const int per = U * a.rp;
  if (QUANT)
    for (int i = threadIdx.x; i < per; i += blockDim.x) top[i] = 0u;
  float ga[8], be[8], mu[8], is[8];
  if (work) {
    gn_params<VEC>(a.gamma, 1.0f, c, a.C, ga);
    gn_params<VEC>(a.beta, 0.0f, c, a.C, be);
    gn_params<VEC>(QUANT ? a.inv_s : nullptr, 1.0f, c, a.C, is);
  }
  griddep_wait();
  griddep_launch_dependents();
  // 8 lanes a group: a warp merges four groups at a time
  const float2* part = a.part + (int64_t)b * a.parts * a.G;
  for (int g0 = 4 * (threadIdx.x >> 5); g0 < a.G; g0 += 4 * (blockDim.x >> 5)) {
    const int g = g0 + (lane >> 3);
    const float2 st = gn_merge(part + min(g, a.G - 1), a.G, a.parts, a.part_rows, a.S, cg, lane & 7, 8);
    if (g < a.G && (lane & 7) == 0) stat[g] = make_float2(st.x, __frsqrt_rn(st.y + a.eps));
  }
  __syncthreads();
  if (work) {
    int g = c / cg, left = cg - c % cg;                  // the vector's channels, group by group
    float2 st = stat[g];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (left == 0 && c + i < a.C) {
        st = stat[++g];
        left = cg;
      }
      --left;
      mu[i] = st.x;
      ga[i] *= st.y;
    }
  }
  const T* X = static_cast<const T*>(a.X) + (int64_t)b * a.S * a.ldx;
  T* Y = static_cast<T*>(a.Y) + (QUANT ? 0 : (int64_t)b * a.S * a.ldy);
  const auto value = [&](const uint32_t(&w)[W], float(&y)[8]) {
    Elem<T>::unpack(w, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fmaf(y[i] - mu[i], ga[i], be[i]);
    gn_act(y, a.act);
  };
  // lanes of this warp that hold the same row as this one
  const uint32_t mates = QUANT ? __match_any_sync(0xFFFFFFFFu, slot) : 0u;
  int buf = 0;
  // rows from the last to the first, U a thread at a time (uniform over the block)
  for (int r0 = hi - 1; r0 >= lo; r0 -= per) {
    uint32_t x[U][W];
    if (work) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 - u * a.rp - slot;
        if (r >= lo) gn_load<T, VEC>(X + (int64_t)r * a.ldx, c, a.C, x[u]);
      }
    }
    if constexpr (!QUANT) {
      if (work) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = r0 - u * a.rp - slot;
          if (r < lo) continue;
          float y[8];
          value(x[u], y);
          T* out = Y + (int64_t)r * a.ldy + c;
          if constexpr (VEC) {
            uint32_t o[W];
            Elem<T>::pack(y, o);
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
              const uint4 d = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
              if (a.streaming) __stcs(reinterpret_cast<uint4*>(out) + i, d);
              else reinterpret_cast<uint4*>(out)[i] = d;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c + i < a.C) out[i] = Elem<T>::from_f32(y[i]);
          }
        }
      }
    } else {
      // Maxima of this step in buffer buf; the next step's buffer is cleared here, two barriers after its last use.
      uint32_t* now = top + buf * per;
      const int nb = buf == 2 ? 0 : buf + 1;
      for (int i = threadIdx.x; i < per; i += blockDim.x) top[nb * per + i] = 0u;
      float y[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 - u * a.rp - slot;
        uint32_t m = 0u;
        if (work && r >= lo) {
          value(x[u], y[u]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            y[u][i] = __fmul_rn(y[u][i], is[i]);
            m = umax(m, abs_bits(y[u][i]));                  // C % 16 == 0: whole vectors
          }
        }
        m = __reduce_max_sync(mates, m);
        if (work && r >= lo && lane == __ffs(mates) - 1) atomicMax(now + u * a.rp + slot, m);
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 - u * a.rp - slot;
        if (work && r >= lo) {
          float scale, mul;
          i8_scale(now[u * a.rp + slot], scale, mul);
          const int64_t row = (int64_t)b * a.S + r;
          if (v == 0) a.sx[row] = scale;
          const float one[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
          const uint2 code = i8_codes(y[u], one, mul);
          *reinterpret_cast<uint2*>(a.Xq + row * a.C + c) = mul == 0.0f ? make_uint2(0u, 0u) : code;
        }
      }
      buf = nb;
    }
  }
}

// Where a sample has many blocks and many groups: their partials merged once, to one entry per group, which the
// second pass then reads as a single block's.  A warp per (sample, group).
__global__ void __launch_bounds__(256) k_group_merge(const float2* part, int64_t BG, int G, int P, int rows, int S,
                                                     int cg, float2* out) {
  griddep_wait();
  const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= BG) return;
  const float2 st = gn_merge(part + i / G * P * G + i % G, G, P, rows, S, cg, threadIdx.x & 31, 32);
  if ((threadIdx.x & 31) == 0) out[i] = make_float2(st.x, st.y * ((float)S * (float)cg));
}

}  // namespace svdq
