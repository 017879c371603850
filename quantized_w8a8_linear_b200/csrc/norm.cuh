// norm.cuh -- layer norm in front of the projections, and its backward pass.
//
//   mean = sum_k x / K,  var = sum_k (x - mean)^2 / K,  rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) * rstd,  y = xh * gamma + beta
//   backward: d = dy * gamma
//             dx = rstd * (d - mean_k(d) - xh * mean_k(d * xh))
//             dgamma = sum_rows dy * xh,  dbeta = sum_rows dy
//
// Both passes are bound by HBM: each row is read once, into shared memory by
// 16-byte cp.async copies that every thread makes for itself (a thread reads
// back only its own slots, so the ring needs no barrier), NORM_STAGES rows
// ahead of the one being reduced. Statistics and sums are fp32; the variance
// is summed from the differences, not from the squares, so a large mean costs
// no bits.
#pragma once
#include "common.cuh"

namespace qlin {

constexpr int NORM_MAX_THREADS = 512;   // 16 warps a row at most
constexpr int NORM_STAGES = 3;

enum NormOut { NORM_OUT_16 = 0, NORM_OUT_E4M3 = 1, NORM_OUT_E4M3_STATIC = 2, NORM_OUT_INT8 = 3 };

struct NormArgs {
  int64_t M, K;
  const uint16_t* X;
  const uint16_t* gamma;   // nullable
  const uint16_t* beta;    // nullable
  float eps;
  void* Y;                 // 16-bit [M,K], or 8-bit codes [M,K]
  float* mean;             // [M], nullable
  float* rstd;             // [M], nullable
  float* s_x;              // [M] per-token scales (dynamic codes)
  const float* x_scale;    // [1] static scale
};

// Sum (or maximum) over the CTA, the same value in every thread and in a
// fixed order. Consecutive calls alternate between two rows of `red`, so one
// barrier a call is enough: a row is written again only after every thread
// has passed the next call's barrier, behind its reads of this one.
template <bool MAX>
__device__ __forceinline__ float cta_reduce(float v, float (*red)[16], int& slot) {
  v = MAX ? warp_max(v) : warp_sum(v);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[slot][warp] = v;
  __syncthreads();
  float t = (lane & 15) < warps ? red[slot][lane & 15] : (MAX ? -INFINITY : 0.0f);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, t, o);
    t = MAX ? fmaxf(t, u) : t + u;
  }
  slot ^= 1;
  return t;
}

// One row at a time per CTA, V 16-byte vectors of it per thread; the CTAs
// stride over the rows. gamma and beta stay in registers when a thread holds
// at most four vectors of them.
template <typename T, int V, int OUT>
__global__ void __launch_bounds__(NORM_MAX_THREADS) k_norm_fwd(const NormArgs a) {
  extern __shared__ uint4 norm_ring[];   // [NORM_STAGES][V][threads]
  __shared__ float red[2][16];
  constexpr bool HOLD = V <= 4;
  const int nt = blockDim.x, tid = threadIdx.x;
  const int KV = static_cast<int>(a.K / 8);
  const int64_t step = gridDim.x;
  int slot = 0;

  auto fetch = [&](int64_t row, int st) {
    if (row < a.M) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int v = j * nt + tid;
        cp_async16(&norm_ring[(st * V + j) * nt + tid], a.X + row * a.K + 8 * static_cast<int64_t>(v), v < KV);
      }
    }
    cp_async_commit();
  };
  auto affine = [&](const uint16_t* p, int j, float none) {
    const int v = j * nt + tid;
    const uint32_t n2 = pack2<T>(none, none);
    return p != nullptr && v < KV ? *reinterpret_cast<const uint4*>(p + 8 * v) : make_uint4(n2, n2, n2, n2);
  };
  for (int i = 0; i < NORM_STAGES - 1; ++i) fetch(blockIdx.x + i * step, i);
  uint4 g[HOLD ? V : 1], b[HOLD ? V : 1];
  if constexpr (HOLD) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      g[j] = affine(a.gamma, j, 1.0f);
      b[j] = affine(a.beta, j, 0.0f);
    }
  }
  float inv_static = 0.0f;
  if constexpr (OUT == NORM_OUT_E4M3_STATIC) inv_static = 1.0f / __ldg(a.x_scale);
  const float rK = 1.0f / static_cast<float>(a.K);

  int st = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += step) {
    fetch(row + (NORM_STAGES - 1) * step, st == 0 ? NORM_STAGES - 1 : st - 1);
    cp_async_wait<NORM_STAGES - 1>();
    uint4 x[V];
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      x[j] = j * nt + tid < KV ? norm_ring[(st * V + j) * nt + tid] : make_uint4(0, 0, 0, 0);
      float f[8];
      widen8<T>(x[j], f);
      s += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
    }
    const float mean = cta_reduce<false>(s, red, slot) * rK;
    float q = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float f[8];
      widen8<T>(x[j], f);
      float d = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) d = fmaf(f[i] - mean, f[i] - mean, d);
      if (j * nt + tid < KV) q += d;
    }
    const float var = cta_reduce<false>(q, red, slot) * rK;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (tid == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    auto value = [&](int j, float (&f)[8]) {
      widen8<T>(x[j], f);
      float gf[8], bf[8];
      widen8<T>(HOLD ? g[HOLD ? j : 0] : affine(a.gamma, j, 1.0f), gf);
      widen8<T>(HOLD ? b[HOLD ? j : 0] : affine(a.beta, j, 0.0f), bf);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = fmaf((f[i] - mean) * rstd, gf[i], bf[i]);
    };
    if constexpr (OUT == NORM_OUT_16) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int v = j * nt + tid;
        float f[8];
        value(j, f);
        if (v < KV) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.Y) + row * a.K + 8 * static_cast<int64_t>(v)) = narrow8<T>(f);
      }
    } else {
      float inv = inv_static;
      if constexpr (OUT != NORM_OUT_E4M3_STATIC) {
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float f[8];
          value(j, f);
          if (j * nt + tid < KV) {
#pragma unroll
            for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
          }
        }
        const float sx = cta_reduce<true>(m, red, slot) / (OUT == NORM_OUT_INT8 ? 127.0f : 448.0f);
        inv = 1.0f / sx;
        if (tid == 0) a.s_x[row] = sx;
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int v = j * nt + tid;
        float f[8];
        value(j, f);
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (OUT == NORM_OUT_INT8) {
            w[h] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[h] |= static_cast<uint32_t>(q_int(f[4 * h + i], inv, 127) & 0xFF) << (8 * i);
          } else {
            w[h] = e4m3x2(q_e4m3_in(f[4 * h], inv), q_e4m3_in(f[4 * h + 1], inv)) |
                   e4m3x2(q_e4m3_in(f[4 * h + 2], inv), q_e4m3_in(f[4 * h + 3], inv)) << 16;
          }
        }
        if (v < KV)
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.Y) + row * a.K + 8 * static_cast<int64_t>(v)) = make_uint2(w[0], w[1]);
      }
    }
    if (++st == NORM_STAGES) st = 0;
  }
  cp_async_wait<0>();
}

struct NormBwdArgs {
  int64_t M, K;
  const uint16_t* dY;
  const uint16_t* X;
  const uint16_t* gamma;   // nullable
  const float* mean;       // [M]
  const float* rstd;       // [M]
  uint16_t* dX;            // [M,K]
  float* part;             // [CTAs][2][K] column sums of each CTA, or nullptr
};

// The two row sums need no second pass: with mean and rstd given, sum d and
// sum d * xh are reduced behind one barrier. Each thread keeps the column
// sums of its own 8 V columns in registers over all rows of its CTA and
// writes them once at the end, for k_norm_bwd_cols to add in CTA order.
template <typename T, int V, bool COLS>
__global__ void __launch_bounds__(NORM_MAX_THREADS) k_norm_bwd(const NormBwdArgs a) {
  extern __shared__ uint4 norm_ring[];   // [NORM_STAGES][2 V][threads]: x, dy
  __shared__ float2 red[2][16];
  const int nt = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = nt >> 5;
  const int KV = static_cast<int>(a.K / 8);
  const int64_t step = gridDim.x;
  auto fetch = [&](int64_t row, int st) {
    if (row < a.M) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int v = j * nt + tid;
        const int64_t at = row * a.K + 8 * static_cast<int64_t>(v);
        cp_async16(&norm_ring[(st * 2 * V + j) * nt + tid], a.X + at, v < KV);
        cp_async16(&norm_ring[(st * 2 * V + V + j) * nt + tid], a.dY + at, v < KV);
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < NORM_STAGES - 1; ++i) fetch(blockIdx.x + i * step, i);
  uint4 g[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int v = j * nt + tid;
    const uint32_t one = pack2<T>(1.0f, 1.0f);
    g[j] = a.gamma != nullptr && v < KV ? *reinterpret_cast<const uint4*>(a.gamma + 8 * v) : make_uint4(one, one, one, one);
  }
  float dg[COLS ? 8 * V : 1] = {}, db[COLS ? 8 * V : 1] = {};
  const float rK = 1.0f / static_cast<float>(a.K);
  int st = 0, slot = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += step) {
    const float mean = __ldg(a.mean + row), rstd = __ldg(a.rstd + row);
    fetch(row + (NORM_STAGES - 1) * step, st == 0 ? NORM_STAGES - 1 : st - 1);
    cp_async_wait<NORM_STAGES - 1>();
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (j * nt + tid < KV) {
        float x[8], dy[8], gf[8];
        widen8<T>(norm_ring[(st * 2 * V + j) * nt + tid], x);
        widen8<T>(norm_ring[(st * 2 * V + V + j) * nt + tid], dy);
        widen8<T>(g[j], gf);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = (x[i] - mean) * rstd, d = dy[i] * gf[i];
          s1 += d;
          s2 = fmaf(d, xh, s2);
          if constexpr (COLS) {
            dg[8 * j + i] = fmaf(dy[i], xh, dg[8 * j + i]);
            db[8 * j + i] += dy[i];
          }
        }
      }
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (warps > 1) {
      if (lane == 0) red[slot][warp] = make_float2(s1, s2);
      __syncthreads();
      const float2 t = (lane & 15) < warps ? red[slot][lane & 15] : make_float2(0.0f, 0.0f);
      s1 = t.x;
      s2 = t.y;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        s1 += __shfl_xor_sync(0xffffffffu, s1, o);
        s2 += __shfl_xor_sync(0xffffffffu, s2, o);
      }
      slot ^= 1;   // as in cta_reduce: one barrier a row, two rows of partial sums
    }
    const float m1 = s1 * rK, m2 = s2 * rK;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = j * nt + tid;
      if (v < KV) {
        float x[8], dy[8], gf[8], o[8];
        widen8<T>(norm_ring[(st * 2 * V + j) * nt + tid], x);
        widen8<T>(norm_ring[(st * 2 * V + V + j) * nt + tid], dy);
        widen8<T>(g[j], gf);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = (x[i] - mean) * rstd;
          o[i] = rstd * (fmaf(dy[i], gf[i], -m1) - xh * m2);
        }
        *reinterpret_cast<uint4*>(a.dX + row * a.K + 8 * static_cast<int64_t>(v)) = narrow8<T>(o);
      }
    }
    if (++st == NORM_STAGES) st = 0;
  }
  cp_async_wait<0>();
  if constexpr (COLS) {
    float* p = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.K;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = j * nt + tid;
      if (v < KV) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          *reinterpret_cast<float4*>(p + 8 * v + i) = make_float4(dg[8 * j + i], dg[8 * j + i + 1], dg[8 * j + i + 2], dg[8 * j + i + 3]);
          *reinterpret_cast<float4*>(p + a.K + 8 * v + i) = make_float4(db[8 * j + i], db[8 * j + i + 1], db[8 * j + i + 2], db[8 * j + i + 3]);
        }
      }
    }
  }
}

// dgamma and dbeta from the CTAs' column sums: 32 columns a CTA, its 16 warps
// take every 16th partial row each and are added in warp order, so the result
// does not depend on timing. Launched as a programmatic dependent.
template <typename T>
__global__ void __launch_bounds__(512) k_norm_bwd_cols(const float* part, int64_t K, int ctas, uint16_t* dgamma, uint16_t* dbeta) {
  __shared__ float red[16][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;   // < 2 K: K % 16 == 0
  griddep_wait();
  float s = 0.0f;
#pragma unroll 4
  for (int i = warp; i < ctas; i += 16) s += part[static_cast<int64_t>(i) * 2 * K + c];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
    s = red[0][lane];
#pragma unroll
    for (int w = 1; w < 16; ++w) s += red[w][lane];
    uint16_t* out = c < K ? dgamma : dbeta;
    if (out != nullptr) out[c < K ? c : c - K] = from_f<T>(s);
  }
}

}  // namespace qlin
