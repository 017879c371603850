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
// ahead of the one being reduced. Statistics and sums are fp32. The variance
// is summed from the differences, not from the squares, and the forward pass
// takes out what rounding the mean to fp32 has left in them: of a large mean
// only the roundings of its sum remain, and sums of values of one binade have
// none while they fit 24 bits (65536 bf16 values, 8192 fp16 ones). The backward
// pass works from the mean it is given. Measured on 16640 rows of 4096, bf16,
// in a run of such calls: forward 47 us (5.8 TB/s of rows in and out), backward
// 72 us (5.7 TB/s), its column sums another 8. To codes, 4352 rows of 4096: FP8
// with dynamic scales 16.9 us, static 14.1, int8 27 (its quantiser works value
// by value), 16 bits 14.6.
#pragma once
#include "common.cuh"
#include "vec.cuh"

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

// Sum (or maximum of absolute values) over the CTA, the same value in every
// thread and in a fixed order. The maximum is taken of the bit patterns, which
// order like the values and put a NaN above them all: fmaxf would drop it, and
// a row of NaN leave as zeros with a scale of zero. Consecutive calls alternate between two rows of `red`, so one
// barrier a call is enough: a row is written again only after every thread
// has passed the next call's barrier, behind its reads of this one.
template <bool MAX>
__device__ __forceinline__ float cta_reduce(float v, float (*red)[16], int& slot) {
  v = MAX ? __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v))) : warp_sum(v);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[slot][warp] = v;
  __syncthreads();
  float t = (lane & 15) < warps ? red[slot][lane & 15] : 0.0f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, t, o);
    t = MAX ? __uint_as_float(max(__float_as_uint(t), __float_as_uint(u))) : t + u;
  }
  slot ^= 1;
  return t;
}

// 8 16-bit values -> four fp32 pairs: the passes below work on pairs, two IEEE
// operations an instruction (a row of 4096 took 15 instructions an element one
// by one, half of the kernel's time at 4.6 TB/s).
typedef unsigned long long f32x2;
template <typename T>
__device__ __forceinline__ void widen8x2(const uint4& u, f32x2 (&f)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      f[i] = f32x2_of(w[i] << 16, w[i] & 0xFFFF0000u);
    } else {
      f[i] = f32x2_of(__float_as_uint(to_f<T>(static_cast<uint16_t>(w[i]))), __float_as_uint(to_f<T>(static_cast<uint16_t>(w[i] >> 16))));
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 narrow8x2(const f32x2 (&f)[4]) {
  return make_uint4(narrow2<T>(lo_f(f[0]), hi_f(f[0])), narrow2<T>(lo_f(f[1]), hi_f(f[1])), narrow2<T>(lo_f(f[2]), hi_f(f[2])),
                    narrow2<T>(lo_f(f[3]), hi_f(f[3])));
}
__device__ __forceinline__ f32x2 twice(float v) { return f32x2_of(__float_as_uint(v), __float_as_uint(v)); }

// One row at a time per CTA, V 16-byte vectors of it per thread; the CTAs
// stride over the rows. gamma and beta stay in registers (widened up to two
// vectors a thread, as they are up to four).
template <typename T, int V, int OUT, int MAXT>
__global__ void __launch_bounds__(MAXT, 512 / MAXT) k_norm_fwd(const NormArgs a) {
  extern __shared__ uint4 norm_ring[];   // [NORM_STAGES][V][threads]
  __shared__ float red[2][16];
  constexpr bool WIDE = V <= 2, HOLD = V <= 4;
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
    const uint32_t n2 = narrow2<T>(none, none);
    return p != nullptr && v < KV ? *reinterpret_cast<const uint4*>(p + 8 * v) : make_uint4(n2, n2, n2, n2);
  };
  for (int i = 0; i < NORM_STAGES - 1; ++i) fetch(blockIdx.x + i * step, i);
  uint4 g[HOLD && !WIDE ? V : 1], b[HOLD && !WIDE ? V : 1];
  f32x2 gw[WIDE ? V : 1][4], bw[WIDE ? V : 1][4];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if constexpr (WIDE) {
      widen8x2<T>(affine(a.gamma, j, 1.0f), gw[j]);
      widen8x2<T>(affine(a.beta, j, 0.0f), bw[j]);
    } else if constexpr (HOLD) {
      g[j] = affine(a.gamma, j, 1.0f);
      b[j] = affine(a.beta, j, 0.0f);
    }
  }
  float inv_static = 0.0f;
  if constexpr (OUT == NORM_OUT_E4M3_STATIC) inv_static = 1.0f / __ldg(a.x_scale);
  const float fK = static_cast<float>(a.K), rK = 1.0f / fK;

  int st = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += step) {
    fetch(row + (NORM_STAGES - 1) * step, st == 0 ? NORM_STAGES - 1 : st - 1);
    cp_async_wait<NORM_STAGES - 1>();
    f32x2 x[V][4];   // the row, then its differences from the mean
    f32x2 s2 = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      widen8x2<T>(j * nt + tid < KV ? norm_ring[(st * V + j) * nt + tid] : make_uint4(0, 0, 0, 0), x[j]);
      s2 = add_f32x2(s2, add_f32x2(add_f32x2(x[j][0], x[j][1]), add_f32x2(x[j][2], x[j][3])));
    }
    const float sum = cta_reduce<false>(lo_f(s2) + hi_f(s2), red, slot);
    const float mean = sum * rK, left = fmaf(-fK, mean, sum) * rK;   // the mean is mean + left
    const f32x2 minus = twice(-mean);
    f32x2 q2 = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      f32x2 d = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[j][i] = add_f32x2(x[j][i], minus);
        d = fma_f32x2(x[j][i], x[j][i], d);
      }
      if (j * nt + tid < KV) q2 = add_f32x2(q2, d);
    }
    float var = fmaf(-left, left, cta_reduce<false>(lo_f(q2) + hi_f(q2), red, slot) * rK);
    if (var < 0.0f) var = 0.0f;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (tid == 0) {
      if (a.mean != nullptr) a.mean[row] = mean + left;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    const f32x2 r2 = twice(rstd), l2 = twice(-left * rstd);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      f32x2 gj[4], bj[4];
      if constexpr (!WIDE) {
        widen8x2<T>(HOLD ? g[HOLD ? j : 0] : affine(a.gamma, j, 1.0f), gj);
        widen8x2<T>(HOLD ? b[HOLD ? j : 0] : affine(a.beta, j, 0.0f), bj);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j][i] = fma_f32x2(fma_f32x2(x[j][i], r2, l2), WIDE ? gw[WIDE ? j : 0][i] : gj[i], WIDE ? bw[WIDE ? j : 0][i] : bj[i]);
    }
    if constexpr (OUT == NORM_OUT_16) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int v = j * nt + tid;
        if (v < KV) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.Y) + row * a.K + 8 * static_cast<int64_t>(v)) = narrow8x2<T>(x[j]);
      }
    } else {
      float inv = inv_static;
      if constexpr (OUT != NORM_OUT_E4M3_STATIC) {
        uint32_t m = 0;   // the largest |y|, as bits
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (j * nt + tid < KV) {
#pragma unroll
            for (int i = 0; i < 4; ++i) m = max(m, max(__float_as_uint(fabsf(lo_f(x[j][i]))), __float_as_uint(fabsf(hi_f(x[j][i])))));
          }
        }
        const float sx = cta_reduce<true>(__uint_as_float(m), red, slot) / (OUT == NORM_OUT_INT8 ? 127.0f : 448.0f);
        inv = 1.0f / sx;
        if (tid == 0) a.s_x[row] = sx;
      }
      inv = fminf(inv, 3.402823466e38f);   // a zero stays zero where 1 / s overflows; all else saturates either way
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int v = j * nt + tid;
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x2 u = x[j][2 * h], t = x[j][2 * h + 1];
          if constexpr (OUT == NORM_OUT_INT8) {
            w[h] = static_cast<uint32_t>(q_int(lo_f(u), inv, 127) & 0xFF) | static_cast<uint32_t>(q_int(hi_f(u), inv, 127) & 0xFF) << 8 |
                   static_cast<uint32_t>(q_int(lo_f(t), inv, 127) & 0xFF) << 16 | static_cast<uint32_t>(q_int(hi_f(t), inv, 127) & 0xFF) << 24;
          } else {
            const f32x2 y0 = mul_f32x2(u, twice(inv)), y1 = mul_f32x2(t, twice(inv));
            w[h] = e4m3x2(lo_f(y0), hi_f(y0)) | e4m3x2(lo_f(y1), hi_f(y1)) << 16;
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
  int row_threads;         // threads of a row: all of the CTA's, or 32 (each warp a row of its own)
};

// The two row sums need no second pass: with mean and rstd given, sum d and
// sum d * xh are reduced behind one barrier. Each thread keeps the column
// sums of its own 8 V columns in registers over all rows of its CTA and
// writes them once at the end, for k_norm_bwd_cols to add in CTA order. Rows
// of up to 1024 take a warp each, whose column sums the CTA adds first: the
// second kernel then reads a row of sums for each CTA, not for each warp
// (16640 rows of 160: 26 us with a CTA of one warp a row).
// MAXT: the threads of a row at most (256 or 512); 512 of them an SM, so that
// the compiler may spread a row's independent work over 128 registers (left to
// itself, at 110, 16640 rows of 4096 took 87 us instead of 70).
template <typename T, int V, bool COLS, int MAXT>
__global__ void __launch_bounds__(MAXT, 512 / MAXT) k_norm_bwd(const NormBwdArgs a) {
  extern __shared__ uint4 norm_ring[];   // [NORM_STAGES][2 V][threads]: x, dy
  __shared__ float red[2][2][16];
  const int nt = a.row_threads, group = threadIdx.x / nt, tid = threadIdx.x % nt, warp = tid >> 5, lane = tid & 31, warps = nt >> 5;
  const int groups = blockDim.x / nt, bt = blockDim.x;   // groups > 1: one warp each, no barrier in the loop
  const int KV = static_cast<int>(a.K / 8);
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups, row0 = static_cast<int64_t>(blockIdx.x) * groups + group;
  auto fetch = [&](int64_t row, int st) {
    if (row < a.M) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int v = j * nt + tid;
        const int64_t at = row * a.K + 8 * static_cast<int64_t>(v);
        cp_async16(&norm_ring[(st * 2 * V + j) * bt + threadIdx.x], a.X + at, v < KV);
        cp_async16(&norm_ring[(st * 2 * V + V + j) * bt + threadIdx.x], a.dY + at, v < KV);
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < NORM_STAGES - 1; ++i) fetch(row0 + i * step, i);
  // up to two vectors a thread: gamma widened, and a row's xh and d kept from
  // the sums to the output; beyond that both are formed again from the ring
  constexpr bool HOLD = V <= 2;
  uint4 g[HOLD ? 1 : V];
  f32x2 gw[HOLD ? V : 1][4];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int v = j * nt + tid;
    const uint32_t o = narrow2<T>(1.0f, 1.0f);
    const uint4 u = a.gamma != nullptr && v < KV ? *reinterpret_cast<const uint4*>(a.gamma + 8 * v) : make_uint4(o, o, o, o);
    if constexpr (HOLD) widen8x2<T>(u, gw[j]);
    else g[j] = u;
  }
  f32x2 dg[COLS ? V : 1][4] = {}, db[COLS ? V : 1][4] = {};
  const float rK = 1.0f / static_cast<float>(a.K);
  int st = 0, slot = 0;
  // xh and d of vector j; dy on the way
  auto terms = [&](int j, const f32x2& minus, const f32x2& r2, f32x2 (&xh)[4], f32x2 (&d)[4], f32x2 (&dy)[4]) {
    widen8x2<T>(norm_ring[(st * 2 * V + j) * bt + threadIdx.x], xh);
    widen8x2<T>(norm_ring[(st * 2 * V + V + j) * bt + threadIdx.x], dy);
    f32x2 gj[4];
    if constexpr (!HOLD) widen8x2<T>(g[HOLD ? 0 : j], gj);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      xh[i] = mul_f32x2(add_f32x2(xh[i], minus), r2);
      d[i] = mul_f32x2(dy[i], HOLD ? gw[HOLD ? j : 0][i] : gj[i]);
    }
  };
  float next_mean = 0.0f, next_rstd = 0.0f;   // looked up a row ahead
  if (row0 < a.M) {
    next_mean = __ldg(a.mean + row0);
    next_rstd = __ldg(a.rstd + row0);
  }
  for (int64_t row = row0; row < a.M; row += step) {
    const float mean = next_mean, rstd = next_rstd;
    if (row + step < a.M) {
      next_mean = __ldg(a.mean + row + step);
      next_rstd = __ldg(a.rstd + row + step);
    }
    fetch(row + (NORM_STAGES - 1) * step, st == 0 ? NORM_STAGES - 1 : st - 1);
    cp_async_wait<NORM_STAGES - 1>();
    const f32x2 minus = twice(-mean), r2 = twice(rstd);
    f32x2 xh[HOLD ? V : 1][4], d[HOLD ? V : 1][4];
    f32x2 t1 = 0, t2 = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (j * nt + tid < KV) {
        f32x2 dy[4];
        f32x2(&xj)[4] = xh[HOLD ? j : 0];
        f32x2(&dj)[4] = d[HOLD ? j : 0];
        terms(j, minus, r2, xj, dj, dy);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          t1 = add_f32x2(t1, dj[i]);
          t2 = fma_f32x2(dj[i], xj[i], t2);
          if constexpr (COLS) {
            dg[j][i] = fma_f32x2(dy[i], xj[i], dg[j][i]);
            db[j][i] = add_f32x2(db[j][i], dy[i]);
          }
        }
      }
    }
    float s1 = lo_f(t1) + hi_f(t1), s2 = lo_f(t2) + hi_f(t2);
    // both sums in one butterfly: s1 in the lower half of the warp, s2 in the upper
    const bool upper = lane >= 16;
    float t = (upper ? s2 : s1) + __shfl_xor_sync(0xffffffffu, upper ? s1 : s2, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (warps > 1) {
      if ((lane & 15) == 0) red[slot][upper][warp] = t;
      __syncthreads();
      t = (lane & 15) < warps ? red[slot][upper][lane & 15] : 0.0f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      slot ^= 1;   // as in cta_reduce: one barrier a row, two rows of partial sums
    }
    s1 = __shfl_sync(0xffffffffu, t, 0);
    s2 = __shfl_sync(0xffffffffu, t, 16);
    const f32x2 m1 = twice(-s1 * rK), m2 = twice(-s2 * rK);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = j * nt + tid;
      if (v < KV) {
        f32x2 dy[4], o[4];
        f32x2(&xj)[4] = xh[HOLD ? j : 0];
        f32x2(&dj)[4] = d[HOLD ? j : 0];
        if constexpr (!HOLD) terms(j, minus, r2, xj, dj, dy);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = mul_f32x2(r2, fma_f32x2(xj[i], m2, add_f32x2(dj[i], m1)));
        *reinterpret_cast<uint4*>(a.dX + row * a.K + 8 * static_cast<int64_t>(v)) = narrow8x2<T>(o);
      }
    }
    if (++st == NORM_STAGES) st = 0;
  }
  cp_async_wait<0>();
  if constexpr (COLS) {
    float* p = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.K;
    float* mine = p;
    if (groups > 1) {   // the ring's memory, when every warp is done with it: [groups][2][K] fp32, 8 K bytes a warp; a warp's share of the ring, 6 V vectors a lane, is 3 V KB, and K <= 256 V
      __syncthreads();
      mine = reinterpret_cast<float*>(norm_ring) + static_cast<int64_t>(group) * 2 * a.K;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = j * nt + tid;
      if (v < KV) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          *reinterpret_cast<float4*>(mine + 8 * v + 2 * i) = make_float4(lo_f(dg[j][i]), hi_f(dg[j][i]), lo_f(dg[j][i + 1]), hi_f(dg[j][i + 1]));
          *reinterpret_cast<float4*>(mine + a.K + 8 * v + 2 * i) = make_float4(lo_f(db[j][i]), hi_f(db[j][i]), lo_f(db[j][i + 1]), hi_f(db[j][i + 1]));
        }
      }
    }
    if (groups > 1) {
      __syncthreads();
      for (int c = threadIdx.x; c < 2 * a.K; c += bt) {
        float t = 0.0f;
        for (int g0 = 0; g0 < groups; ++g0) t += reinterpret_cast<const float*>(norm_ring)[static_cast<int64_t>(g0) * 2 * a.K + c];
        p[c] = t;
      }
    }
  }
}

// dgamma and dbeta from the CTAs' column sums: 128 columns a CTA, its 16 warps
// take every 16th partial row each and are added in warp order, so the result
// does not depend on timing. Launched as a programmatic dependent.
template <typename T>
__global__ void __launch_bounds__(512) k_norm_bwd_cols(const float* part, int64_t K, int ctas, uint16_t* dgamma, uint16_t* dbeta) {
  __shared__ float4 red[16][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 128 + 4 * lane;   // K % 16 == 0: a thread's columns are of one kind
  griddep_wait();
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < 2 * K) {
#pragma unroll 8
    for (int i = warp; i < ctas; i += 16) {
      const float4 v = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(i) * 2 * K + c);
      s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
    }
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < 2 * K) {
#pragma unroll
    for (int w = 1; w < 16; ++w) {
      const float4 v = red[w][lane];
      s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
    }
    uint16_t* out = c < K ? dgamma : dbeta;
    if (out != nullptr) *reinterpret_cast<uint2*>(out + (c < K ? c : c - K)) = make_uint2(narrow2<T>(s.x, s.y), narrow2<T>(s.z, s.w));
  }
}

}  // namespace qlin
