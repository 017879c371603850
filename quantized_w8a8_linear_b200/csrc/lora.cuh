// lora.cuh -- low-rank adapters of many requests beside a shared projection,
// and their gradients.
//
//   a = idx[m]:  H[m] = X[m] A[a]^T,   Y[m] += s[a] H[m] B[a]^T
//   backward:    dH[m] = s[a] dY[m] B[a],           dX[m] += dH[m] A[a]
//                dA[a] = sum_m dH[m]^T X[m],        dB[a] = s[a] sum_m dY[m]^T H[m]
//
// X [M,K], Y [M,N], A [L,R,K], B [L,N,R] 16-bit, H and dH [M,R] fp32.
//
// A plan sorts the rows by adapter once per batch (k_lora_plan): tiles of up
// to 128 rows of one adapter, as lists of row numbers. Every kernel works on
// tiles, so each row meets its own adapter only, whatever the order of the
// rows, and gathers them with TMA (tile::gather4: four rows of 128 bytes an
// instruction; a row number past the tensor reads as zeros). The products are
// thin (R <= 128), so all three kernels are bound by the 16-bit matrices they
// read and write, not by the tensor cores:
//   k_lora_shrink  H or dH: contraction over K or N;
//   k_lora_expand  Y or dX: contraction over R;
//   k_lora_wgrad   dA and dB: contraction over the rows of an adapter.
//
// H enters the second product as two 16-bit parts, hi = T(h) and
// lo = T(h - hi), two MMAs on one staged operand: 16 (bf16) or 22 (fp16)
// significant bits, where hi alone would add an error of the size of the
// output's own rounding. fp16 parts are taken of h / 2^e with 2^e the largest
// power of two in the row (exact), so neither overflow nor subnormals cut them.
//
// All mbarrier waits are bounded (common.cuh).
#pragma once
#include "common.cuh"

namespace qlin {

constexpr int LORA_TILE = 128;       // rows of a tile
constexpr int LORA_BK = 64;          // 16-bit elements of a 128-byte swizzled row
constexpr int LORA_MAX_R = 128;
constexpr int LORA_MAX_L = 1024;

// ---------------------------------------------------------------------------
// plan: int32 words
//   [0] M  [1] L  [2] tiles  [3..15] 0
//   tile0 [L + 1]       first tile of each adapter (tile0[L] = tiles)
//   info  [Tmax][2]     adapter and row count of a tile
//   rows  [Tmax][128]   row numbers, in row order; M past the count
// Tmax = M / 128 + min(L, M) bounds the sum of ceil(rows / 128) over adapters.
// ---------------------------------------------------------------------------
__host__ __device__ inline int64_t lora_max_tiles(int64_t M, int64_t L) { return M / LORA_TILE + (L < M ? L : M); }
__host__ __device__ inline int64_t lora_info_at(int64_t L) { return 16 + (L + 4) / 4 * 4; }
__host__ __device__ inline int64_t lora_rows_at(int64_t M, int64_t L) { return lora_info_at(L) + (2 * lora_max_tiles(M, L) + 3) / 4 * 4; }
__host__ __device__ inline int64_t lora_plan_words(int64_t M, int64_t L) { return lora_rows_at(M, L) + LORA_TILE * lora_max_tiles(M, L); }

struct LoraPlan {
  const int* w;
  int64_t M, L;
  __device__ __forceinline__ const int* tile0() const { return w + 16; }
  __device__ __forceinline__ int2 info(int t) const { return *reinterpret_cast<const int2*>(w + lora_info_at(L) + 2 * static_cast<int64_t>(t)); }
  __device__ __forceinline__ const int* rows(int t) const { return w + lora_rows_at(M, L) + static_cast<int64_t>(LORA_TILE) * t; }
  // Tiles of the plan; 0, with QLIN_ERR_INVALID_ARG in the status word, when
  // the buffer holds another problem's plan (its row numbers are not used).
  __device__ __forceinline__ int tiles() const {
    const int4 h = *reinterpret_cast<const int4*>(w);
    if (h.x == static_cast<int>(M) && h.y == static_cast<int>(L) && h.z >= 0 && h.z <= lora_max_tiles(M, L)) return h.z;
    atomicExch(&g_status, 1 /* QLIN_ERR_INVALID_ARG */);
    return 0;
  }
};

constexpr int LORA_PLAN_THREADS = 1024;

// Stable counting sort of the rows by adapter, in one CTA: warp w counts the
// adapters of its contiguous share of the rows, a scan over (adapter, warp)
// turns the counts into places, and the warps walk their shares again, each
// row's place within 32 rows from the ballot of its equals. No atomics, so
// the order (and every sum over it) is the same in every run.
__global__ void __launch_bounds__(LORA_PLAN_THREADS) k_lora_plan(const int* idx, int64_t M, int64_t L64, int* plan) {
  extern __shared__ int lora_count[];   // [32][L]
  __shared__ int warp_total[32];
  const int L = static_cast<int>(L64);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t per = (M + 1023) / 1024 * 32;
  const int64_t lo = warp * per < M ? warp * per : M, hi = lo + per < M ? lo + per : M;
  int* tile0 = plan + 16;
  int* info = plan + lora_info_at(L);
  int* rows = plan + lora_rows_at(M, L);
  for (int i = tid; i < 32 * L; i += LORA_PLAN_THREADS) lora_count[i] = 0;
  __syncthreads();
  int* mine = lora_count + warp * L;
  auto adapter = [&](int64_t m) {
    const int a = m < hi ? idx[m] : -1;
    return a >= 0 && a < L ? a : -1;
  };
  for (int64_t m0 = lo; m0 < hi; m0 += 32) {
    const int a = adapter(m0 + lane);
    const uint32_t same = __match_any_sync(0xffffffffu, a);
    if (a >= 0 && lane == __ffs(same) - 1) mine[a] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // thread a: rows of adapter a, and the places of its rows within them
  int n = 0;
  if (tid < L) {
    for (int w = 0; w < 32; ++w) {
      const int c = lora_count[w * L + tid];
      lora_count[w * L + tid] = n;
      n += c;
    }
  }
  const int tiles = (n + LORA_TILE - 1) / LORA_TILE;
  int scan = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += u;
  }
  if (lane == 31) warp_total[warp] = scan;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += warp_total[w];
  const int first = before + scan - tiles;
  if (tid < L) {
    tile0[tid] = first;
    if (tid == L - 1) tile0[L] = first + tiles;
    for (int t = 0; t < tiles; ++t) {
      info[2 * (first + t)] = tid;
      info[2 * (first + t) + 1] = n - t * LORA_TILE < LORA_TILE ? n - t * LORA_TILE : LORA_TILE;
    }
    for (int i = n; i < tiles * LORA_TILE; ++i) rows[static_cast<int64_t>(first) * LORA_TILE + i] = static_cast<int>(M);
    for (int w = 0; w < 32; ++w) lora_count[w * L + tid] += first * LORA_TILE;
  }
  if (tid < 16) {
    int total = 0;
    for (int w = 0; w < 32; ++w) total += warp_total[w];
    plan[tid] = tid == 0 ? static_cast<int>(M) : tid == 1 ? L : tid == 2 ? total : 0;
  }
  __syncthreads();
  for (int64_t m0 = lo; m0 < hi; m0 += 32) {
    const int a = adapter(m0 + lane);
    const uint32_t same = __match_any_sync(0xffffffffu, a);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (a >= 0) rows[mine[a] + rank] = static_cast<int>(m0 + lane);
    __syncwarp();
    if (a >= 0 && rank == 0) mine[a] += __popc(same);
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// helpers
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tma_gather4(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t x, const int4& r) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// MN-major operand tile in the 128-byte swizzle: one 128-byte row (64 elements
// of M or N) per step of the contraction, 8-row groups 1024 bytes apart
// (stride byte offset), the next 64 elements of M or N `next` bytes on
// (leading byte offset). 16 steps of the contraction are 2048 bytes.
__device__ __forceinline__ uint64_t sdesc_mn128(uint32_t saddr, uint32_t next) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((next & 0x3FFFFu) >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
// bits 15 and 16 of the instruction descriptor: A and B are MN-major
constexpr uint32_t IDESC_A_MN = 1u << 15, IDESC_B_MN = 1u << 16;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t saddr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(saddr), "r"(rank)
      : "memory");
  return v;
}

// Waits (bounded) for the copies a producer that gave up still has in flight:
// the ring slots before `stage` in issue order, as far as they were used.
__device__ __forceinline__ void drain_ring(uint64_t* full_bar, int stages, int stage, uint32_t phase, uint32_t issued) {
  for (int i = 0; i < stages; ++i) {
    if (--stage < 0) { stage = stages - 1; phase ^= 1u; }
    if (issued & (1u << stage)) {
      const uint32_t a = smem_u32(&full_bar[stage]);
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(a, phase) && globaltimer() - t0 < drain_limit_ns()) {}
    }
  }
}

// Waits (bounded) for the MMAs this thread issued, before TMEM is freed.
__device__ __forceinline__ void drain_mma(uint64_t* bar) {
  umma_commit(bar);
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(a, 0) && globaltimer() - t0 < drain_limit_ns()) {}
}

// 8 fp32 values -> two 16-byte chunks of 16-bit values, hi + lo = the value to
// 16 (bf16) or 22 (fp16) bits. Where hi is not finite lo is 0, so an infinite
// or NaN value stays what it is.
template <typename T>
__device__ __forceinline__ void split8(const float (&f)[8], uint4& hi, uint4& lo) {
  uint16_t h[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = from_f<T>(f[i]);
    const float r = f[i] - to_f<T>(h[i]);
    l[i] = fabsf(r) <= fabsf(f[i]) ? from_f<T>(r) : static_cast<uint16_t>(0);   // false for NaN and for hi = inf
  }
  hi = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
  lo = make_uint4(l[0] | (l[1] << 16), l[2] | (l[3] << 16), l[4] | (l[5] << 16), l[6] | (l[7] << 16));
}

// ---------------------------------------------------------------------------
// k_lora_shrink: H[rows of the tile] = X W^T (c partial sums over the
// contraction, one per CTA of a cluster).
//   W_MN 0: W = A[a] [R, K], K-major;   1: W = B[a] [N, R] read as its
//   transpose, MN-major, with X = dY and the contraction over N.
// A cluster of c CTAs shares a tile, each with 1/c of the contraction; the
// fp32 partial tiles meet in shared memory and CTA q adds rows q, q + c, ...
// of all of them in rank order (distributed shared memory; no workspace and
// no second kernel). c is chosen so that few tiles still fill the SMs.
// ---------------------------------------------------------------------------
constexpr int LORA_SHRINK_THREADS = 192;   // warp 0 TMA, warp 1 MMA, warps 2-5 epilogue

struct LoraShrinkParams {
  LoraPlan plan;
  int64_t C;            // contraction length (K, or N)
  int R;
  const float* scale;   // [L], or nullptr: 1
  float* H;             // [M,R]
};

template <int RB>   // ceil(R / 64)
struct LoraShrinkSmem {
  static constexpr int STAGES = 4;
  static constexpr int A_BYTES = LORA_TILE * 128;
  static constexpr int W_BYTES = RB * 64 * 128;
  static constexpr int STAGE_BYTES = A_BYTES + W_BYTES;
  static constexpr int BAR_BYTES = 8 * (2 * STAGES + 2) + 16;
  static constexpr int TOTAL = 1024 + STAGES * STAGE_BYTES + BAR_BYTES;
  // the partial tile takes the stages' place after the last MMA
  static_assert(LORA_TILE * (RB * 64 + 4) * 4 <= STAGES * STAGE_BYTES, "partial tile");
};

template <typename T, int RB, bool W_MN>
__global__ void __launch_bounds__(LORA_SHRINK_THREADS)
    k_lora_shrink(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const LoraShrinkParams p,
                  const int cluster) {
  using S = LoraShrinkSmem<RB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto sA = [&](int s) { return smem + s * S::STAGE_BYTES; };
  auto sW = [&](int s) { return smem + s * S::STAGE_BYTES + S::A_BYTES; };
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + S::STAGES * S::STAGE_BYTES);
  uint64_t* empty_bar = full_bar + S::STAGES;
  uint64_t* tfull_bar = empty_bar + S::STAGES;
  uint64_t* drain_bar = tfull_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr uint32_t TCOLS = RB * 64;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(tfull_bar, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // X, the plan and H's earlier readers belong to kernels before this one
  griddep_wait();
  griddep_launch_dependents();

  const int tile = blockIdx.x / cluster;
  const int rank = cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
  const bool work = tile < p.plan.tiles();   // the same in all CTAs of the cluster
  const int2 info = work ? p.plan.info(tile) : make_int2(0, 0);
  const int a = info.x, n = info.y;
  const int kbs = static_cast<int>((p.C + LORA_BK - 1) / LORA_BK);
  const int kb0 = static_cast<int>(static_cast<int64_t>(kbs) * rank / cluster);
  const int kb1 = static_cast<int>(static_cast<int64_t>(kbs) * (rank + 1) / cluster);
  const int Rp = (p.R + 15) / 16 * 16;

  if (work && warp == 0) {
    // ---------------- TMA producer: lane i gathers rows 4 i .. 4 i + 3 ----------------
    const int groups = (n + 3) / 4;
    const int4 r4 = reinterpret_cast<const int4*>(p.plan.rows(tile))[lane];
    const uint32_t bytes = static_cast<uint32_t>(groups * 512 + (W_MN ? RB * 64 : Rp) * 128);
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool good = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (lane == 0) {
        good = mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag);
        if (good) mbar_arrive_expect_tx(&full_bar[stage], bytes);
      }
      good = __shfl_sync(0xffffffffu, good, 0);
      if (!good) break;
      if (lane < groups) tma_gather4(sA(stage) + lane * 512, &tmX, &full_bar[stage], kb * LORA_BK, r4);
      if (lane == 0) {
        if constexpr (W_MN) {
#pragma unroll
          for (int b = 0; b < RB; ++b) tma_load_3d(sW(stage) + b * 8192, &tmW, &full_bar[stage], b * 64, kb * LORA_BK, a);
        } else {
          tma_load_3d(sW(stage), &tmW, &full_bar[stage], kb * LORA_BK, 0, a);
        }
      }
      issued |= 1u << stage;
      if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
    }
    if (!good && lane == 0) drain_ring(full_bar, S::STAGES, stage, phase, issued);
  } else if (work && warp == 1) {
    if (lane == 0) {
      // ---------------- MMA issuer ----------------
      constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
      const uint32_t idesc = W_MN ? (idesc_f16(LORA_TILE, RB * 64, bf) | IDESC_B_MN) : idesc_f16(LORA_TILE, Rp, bf);
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&full_bar[stage], phase, abort_flag)) break;
        tc_fence_after();
        const uint64_t adesc = sdesc_k128(smem_u32(sA(stage)));
        const uint64_t bdesc = W_MN ? sdesc_mn128(smem_u32(sW(stage)), 8192u) : sdesc_k128(smem_u32(sW(stage)));
#pragma unroll
        for (int k = 0; k < LORA_BK / 16; ++k)
          umma<2>(tmem_base, adesc + 2u * k, bdesc + (W_MN ? 128u : 2u) * k, idesc, (kb != kb0 || k != 0) ? 1u : 0u);
        umma_commit(&empty_bar[stage]);
        if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
      }
      umma_commit(tfull_bar);
      drain_mma(drain_bar);
    }
  } else if (work) {
    // ---------------- epilogue: row q * 32 + lane of the tile ----------------
    const int q = warp & 3;
    const int r = q * 32 + lane;
    const bool good = mbar_wait(tfull_bar, 0, abort_flag) && kb1 > kb0;
    tc_fence_after();
    const float s = p.scale != nullptr ? __ldg(p.scale + a) : 1.0f;
    float* out = cluster > 1 ? reinterpret_cast<float*>(smem) + r * (Rp + 4)
                             : p.H + static_cast<int64_t>(r < n ? p.plan.rows(tile)[r] : 0) * p.R;
    if (q * 32 < n) {
      for (int c = 0; c < p.R; c += 16) {
        uint32_t v[16];
        __syncwarp();
        tmem_ld16(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + c, v);
        tmem_wait16(v);
        if (r < n) {
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            if (c + i < p.R) {
              float4 f = make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]), __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
              if (!good) f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              if (cluster == 1) f = make_float4(f.x * s, f.y * s, f.z * s, f.w * s);
              *reinterpret_cast<float4*>(out + c + i) = f;
            }
          }
        }
      }
    }
    tc_fence_before();
  }
  if (cluster > 1) {
    cluster_sync();
    if (work) {
      const float s = p.scale != nullptr ? __ldg(p.scale + a) : 1.0f;
      const int r4 = p.R / 4;
      const int mine = rank < n ? (n - rank + cluster - 1) / cluster : 0;   // rows rank, rank + cluster, ...
      const uint32_t base = smem_u32(smem);
      for (int e = threadIdx.x; e < mine * r4; e += LORA_SHRINK_THREADS) {
        const int r = rank + e / r4 * cluster, c = e % r4 * 4;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k = 0; k < cluster; ++k) {
          const float4 f = ld_cluster_f4(base + static_cast<uint32_t>((r * (Rp + 4) + c) * 4), k);
          sum = make_float4(sum.x + f.x, sum.y + f.y, sum.z + f.z, sum.w + f.w);
        }
        *reinterpret_cast<float4*>(p.H + static_cast<int64_t>(p.plan.rows(tile)[r]) * p.R + c) =
            make_float4(sum.x * s, sum.y * s, sum.z * s, sum.w * s);
      }
    }
    cluster_sync();   // no CTA leaves while another reads its partial tile
  }
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, TCOLS);
  }
}

// ---------------------------------------------------------------------------
// k_lora_expand: Y[rows of the tile] += s (hi + lo) V^T, 64 columns a unit.
//   V_MN 0: V = B[a] [N, R], K-major;   1: V = A[a] [R, K] read as its
//   transpose, MN-major, with Y = dX and K columns.
// Persistent: the units (tile, 64 columns), columns fastest, are cut into one
// equal range per CTA, so that every SM moves the same number of bytes
// whatever the tiles; a range spans few tiles, whose H is split into its
// parts once each. Y comes in through TMA gathers beside V, is updated in
// place in shared memory and leaves in 128-byte row pieces. The copies of Y
// and V start before the kernel that makes H has ended (programmatic
// dependent launch); only the readers of H wait for it.
//   VEC false: rows of Y that are not multiples of 16 bytes are read and
//   written two bytes at a time by the epilogue instead.
// ---------------------------------------------------------------------------
constexpr int LORA_EXPAND_THREADS = 192;   // warp 0 TMA, warp 1 MMA, warps 2-5 split H and the epilogue
constexpr int LORA_EXPAND_BN = 64;

struct LoraExpandParams {
  LoraPlan plan;
  int64_t N;            // columns of Y
  int R;
  const float* scale;   // [L], or nullptr: 1
  const float* H;       // [M,R]
  uint16_t* Y;          // [M,N]
};

template <int RB, bool VEC>
struct LoraExpandSmem {
  static constexpr int STAGES = 3;
  static constexpr int H_BYTES = RB * LORA_TILE * 128;                 // one part
  static constexpr int V_BYTES = RB * 64 * 128;
  static constexpr int Y_BYTES = VEC ? LORA_TILE * 128 : 0;
  static constexpr int STAGE_BYTES = V_BYTES + Y_BYTES;
  static constexpr int D_BYTES = VEC ? 0 : LORA_TILE * 65 * 4;         // update staged for the 2-byte path
  static constexpr int BAR_BYTES = 8 * (2 * STAGES + 6) + 16;
  static constexpr int TOTAL = 1024 + 2 * H_BYTES + STAGES * STAGE_BYTES + D_BYTES + BAR_BYTES;
};

template <typename T, int RB, bool V_MN, bool VEC>
__global__ void __launch_bounds__(LORA_EXPAND_THREADS)
    k_lora_expand(const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmY, const LoraExpandParams p) {
  using S = LoraExpandSmem<RB, VEC>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sH = smem;   // [hi, lo][RB][128 rows][128 bytes]
  auto sV = [&](int s) { return smem + 2 * S::H_BYTES + s * S::STAGE_BYTES; };
  auto sY = [&](int s) { return smem + 2 * S::H_BYTES + s * S::STAGE_BYTES + S::V_BYTES; };
  float* sD = reinterpret_cast<float*>(smem + 2 * S::H_BYTES + S::STAGES * S::STAGE_BYTES);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + 2 * S::H_BYTES + S::STAGES * S::STAGE_BYTES + S::D_BYTES);
  uint64_t* empty_bar = full_bar + S::STAGES;
  uint64_t* tfull_bar = empty_bar + S::STAGES;   // [2]
  uint64_t* tempty_bar = tfull_bar + 2;          // [2]
  uint64_t* hfull_bar = tempty_bar + 2;
  uint64_t* drain_bar = hfull_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr uint32_t TCOLS = 2 * LORA_EXPAND_BN;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 4);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], 4);
    }
    mbar_init(hfull_bar, 4);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmV);
    if (VEC) tma_prefetch_desc(&tmY);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int nbs = static_cast<int>((p.N + LORA_EXPAND_BN - 1) / LORA_EXPAND_BN);
  const int64_t units = static_cast<int64_t>(p.plan.tiles()) * nbs;
  const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  const int Rp = (p.R + 15) / 16 * 16;

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    int stage = 0, tile = -1, a = 0, groups = 0;
    int4 r4 = make_int4(0, 0, 0, 0);
    uint32_t phase = 0, issued = 0;
    bool good = true;
    for (int64_t u = u0; u < u1; ++u) {
      const int t = static_cast<int>(u / nbs), n0 = static_cast<int>(u % nbs) * LORA_EXPAND_BN;
      if (t != tile) {
        tile = t;
        const int2 info = p.plan.info(t);
        a = info.x;
        groups = (info.y + 3) / 4;
        r4 = reinterpret_cast<const int4*>(p.plan.rows(t))[lane];
      }
      if (lane == 0) {
        good = mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag);
        if (good) mbar_arrive_expect_tx(&full_bar[stage], static_cast<uint32_t>((V_MN ? Rp * 128 : RB * 8192) + (VEC ? groups * 512 : 0)));
      }
      good = __shfl_sync(0xffffffffu, good, 0);
      if (!good) break;
      if (VEC && lane < groups) tma_gather4(sY(stage) + lane * 512, &tmY, &full_bar[stage], n0, r4);
      if (lane == 0) {
        if constexpr (V_MN) {
          tma_load_3d(sV(stage), &tmV, &full_bar[stage], n0, 0, a);
        } else {
#pragma unroll
          for (int b = 0; b < RB; ++b) tma_load_3d(sV(stage) + b * 8192, &tmV, &full_bar[stage], b * 64, n0, a);
        }
      }
      issued |= 1u << stage;
      if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
    }
    if (!good && lane == 0) drain_ring(full_bar, S::STAGES, stage, phase, issued);
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- MMA issuer ----------------
      constexpr uint32_t idesc = idesc_f16(LORA_TILE, LORA_EXPAND_BN, std::is_same<T, __nv_bfloat16>::value) | (V_MN ? IDESC_B_MN : 0u);
      const int ksteps = Rp / 16;
      int stage = 0, acc = 0, tile = -1;
      uint32_t phase = 0, acc_phase = 0, h_phase = 0;
      for (int64_t u = u0; u < u1; ++u) {
        const int t = static_cast<int>(u / nbs);
        if (t != tile) {
          tile = t;
          if (!mbar_wait(hfull_bar, h_phase, abort_flag)) break;
          h_phase ^= 1u;
        }
        if (!mbar_wait(&tempty_bar[acc], acc_phase ^ 1u, abort_flag)) break;
        if (!mbar_wait(&full_bar[stage], phase, abort_flag)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * LORA_EXPAND_BN);
        const uint32_t v = smem_u32(sV(stage)), h = smem_u32(sH);
        for (int part = 0; part < 2; ++part) {
          for (int k = 0; k < ksteps; ++k) {
            const uint64_t adesc = sdesc_k128(h + part * S::H_BYTES + (k >> 2) * (LORA_TILE * 128)) + 2u * (k & 3);
            const uint64_t bdesc = V_MN ? sdesc_mn128(v, 0u) + 128u * k : sdesc_k128(v + (k >> 2) * 8192) + 2u * (k & 3);
            umma<2>(d, adesc, bdesc, idesc, (part | k) != 0 ? 1u : 0u);
          }
        }
        umma_commit(&tfull_bar[acc]);
        if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      drain_mma(drain_bar);
    }
  } else {
    // ---------------- H's parts, then the epilogue: warp for rows 32 q .. 32 q + 31 ----------------
    const int q = warp & 3;
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    int stage = 0, acc = 0, tile = -1, n = 0, my_row = 0;
    float s = 1.0f;    // scale[a], times the power of two of the lane's row (fp16)
    uint32_t phase = 0, acc_phase = 0;
    bool good = true;
    griddep_wait();    // H
    for (int64_t u = u0; u < u1; ++u) {
      const int t = static_cast<int>(u / nbs);
      const int64_t n0 = (u % nbs) * LORA_EXPAND_BN;
      if (t != tile) {
        // the MMAs that read the previous tile's parts have completed: this
        // warp has waited for the accumulator of its last unit
        tile = t;
        const int2 info = p.plan.info(t);
        n = info.y - q * 32;
        my_row = n > lane ? p.plan.rows(t)[q * 32 + lane] : 0;
        const float sa = p.scale != nullptr ? __ldg(p.scale + info.x) : 1.0f;
        s = sa;
        constexpr int CH = RB * 8;   // 8-value chunks of a row: lanes of a warp that share a row
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int e = i * 32 + lane, r = e / CH, c = e % CH;
          float f[8] = {};
          const int row = __shfl_sync(0xffffffffu, my_row, r);
          if (r < n && 8 * c < p.R) {
            const float4* src = reinterpret_cast<const float4*>(p.H + static_cast<int64_t>(row) * p.R + 8 * c);
            const float4 x = src[0], y = src[1];
            f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
            f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
          }
          if constexpr (std::is_same<T, __half>::value) {
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
#pragma unroll
            for (int o = CH / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            // 2^e <= max < 2^(e+1); rows of zeros, subnormals, infinities keep 1
            const uint32_t eb = __float_as_uint(m) >> 23;
            const bool norm = eb >= 1 && eb <= 253;
            const float up = norm ? __uint_as_float(eb << 23) : 1.0f;
            const float down = norm ? __uint_as_float((254u - eb) << 23) : 1.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= down;
            // the lane whose TMEM row this is keeps 2^e: rows of this step are r of lanes 0, CH, ...
            const float up_mine = __shfl_sync(0xffffffffu, up, (lane % (32 / CH)) * CH);
            if (lane / (32 / CH) == i) s = sa * up_mine;
          }
          uint4 hi, lo;
          split8<T>(f, hi, lo);
          const int rr = q * 32 + r;
          uint8_t* d = sH + (c >> 3) * (LORA_TILE * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4);
          *reinterpret_cast<uint4*>(d) = hi;
          *reinterpret_cast<uint4*>(d + S::H_BYTES) = lo;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(hfull_bar);
      }
      if (VEC) good = mbar_wait(&full_bar[stage], phase, abort_flag);   // Y, written by TMA
      good = good && mbar_wait(&tfull_bar[acc], acc_phase, abort_flag);
      if (!__all_sync(0xffffffffu, good)) break;
      tc_fence_after();
      if (n > 0) {
        uint32_t v[2][32];
        tmem_ld32(lane_base + static_cast<uint32_t>(acc * LORA_EXPAND_BN), v[0]);
        tmem_ld32(lane_base + static_cast<uint32_t>(acc * LORA_EXPAND_BN + 32), v[1]);
        tmem_wait_regs32(v[0]);
        tmem_wait_regs32(v[1]);
        tc_fence_before();
        if constexpr (VEC) {
          const int rr = q * 32 + lane;
          uint8_t* yr = sY(stage) + rr * 128;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint4* at = reinterpret_cast<uint4*>(yr + ((c ^ (rr & 7)) << 4));
            float f[8];
            uint16_t h[8];
            unpack8(*at, h);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = fmaf(__uint_as_float(v[c >> 2][(c & 3) * 8 + i]), s, to_f<T>(h[i]));
            *at = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
          }
          __syncwarp();
          const int c = lane & 7;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3), row = __shfl_sync(0xffffffffu, my_row, r);
            if (r < n && n0 + 8 * c < p.N)
              *reinterpret_cast<uint4*>(p.Y + static_cast<int64_t>(row) * p.N + n0 + 8 * c) =
                  *reinterpret_cast<const uint4*>(sY(stage) + (q * 32 + r) * 128 + ((c ^ (r & 7)) << 4));
          }
        } else {
          float* d = sD + (q * 32) * 65;
#pragma unroll
          for (int i = 0; i < 64; ++i) d[lane * 65 + i] = __uint_as_float(v[i >> 5][i & 31]) * s;
          __syncwarp();
          const int rows = n < 32 ? n : 32;
#pragma unroll 4
          for (int r = 0; r < rows; ++r) {
            uint16_t* y = p.Y + static_cast<int64_t>(__shfl_sync(0xffffffffu, my_row, r)) * p.N + n0;
#pragma unroll
            for (int h = 0; h < 64; h += 32) {
              if (n0 + h + lane < p.N) y[h + lane] = from_f<T>(to_f<T>(y[h + lane]) + d[r * 65 + h + lane]);
            }
          }
          __syncwarp();
        }
      }
      // this warp's generic accesses to the stage come before the next copy into it
      if (VEC) fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&tempty_bar[acc]);
        mbar_arrive(&empty_bar[stage]);
      }
      if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
  }
  __syncthreads();
  griddep_wait();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, TCOLS);
  }
}

// ---------------------------------------------------------------------------
// k_lora_wgrad: D[a][c, r] = sum over the rows m of adapter a of X[m, c] G[m, r]
// for both gradients in one launch: side 0 X, G = dH -> dA [L,R,K];
// side 1 dY, G = H -> s[a] D -> dB [L,N,R].
// A unit is 256 columns of one tile; units run (side, columns, tile) with the
// tile fastest and are cut into one equal range per CTA. The tile of X is the
// A operand and the parts of G the B operand, both MN-major as they lie in
// memory (one 128-byte row per step of the contraction), so nothing is
// transposed. Sums stay in TMEM over the tiles of an adapter. An adapter
// whose tiles are cut between CTAs leaves fp32 partial sums, slot 0 for a
// CTA's first segment if it began before, slot 1 for the last one, and
// k_lora_wgrad_join adds them in CTA order.
// bf16 only: G's parts need fp32's exponent range (a power of two per row, as
// k_lora_expand takes out, does not leave a sum over rows).
// ---------------------------------------------------------------------------
constexpr int LORA_WG_THREADS = 448;   // warp 0 TMA, warp 1 MMA, warps 2-5 epilogue, warps 6-13 split G
constexpr int LORA_WG_CONV_WARPS = 8;
constexpr int LORA_WG_COLS = 256;      // columns of a unit: two MMAs of M = 128

struct LoraWgradParams {
  LoraPlan plan;
  int R, ctas;
  int64_t cols[2];       // K, N
  const float* G[2];     // dH, H [M,R]
  const float* scale;    // [L]
  uint16_t* out[2];      // dA [L,R,K], dB [L,N,R]
  float* part;           // [ctas][2][R][256] fp32
};

// Columns, range and segment arithmetic shared by the kernel and the join.
struct LoraWgradUnits {
  int cg0, cgs, tiles, ctas;
  int64_t units;
  __device__ __forceinline__ LoraWgradUnits(const LoraWgradParams& p) {
    cg0 = static_cast<int>((p.cols[0] + LORA_WG_COLS - 1) / LORA_WG_COLS);
    cgs = cg0 + static_cast<int>((p.cols[1] + LORA_WG_COLS - 1) / LORA_WG_COLS);
    tiles = p.plan.tiles();
    units = static_cast<int64_t>(cgs) * tiles;
    ctas = static_cast<int>(units < p.ctas ? units : p.ctas);   // each has a unit: no slot is read that was not written
  }
  // first unit of a CTA (of the CTAs past the last one with units: `units`), and the CTA of a unit
  __device__ __forceinline__ int64_t first(int64_t cta) const { return cta < ctas ? units * cta / ctas : units; }
  __device__ __forceinline__ int owner(int64_t u) const { return static_cast<int>(((u + 1) * ctas - 1) / units); }
};

template <int RB>
struct LoraWgradSmem {
  static constexpr int STAGES = RB == 1 ? 4 : 3;
  static constexpr int X_BYTES = 2 * LORA_TILE * 128;            // 128 columns of the tile: two 64-column halves
  static constexpr int G_BYTES = RB * LORA_TILE * 128;           // one part
  static constexpr int BAR_BYTES = 8 * (2 * STAGES + 9) + 16;
  static constexpr int TOTAL = 1024 + STAGES * X_BYTES + 4 * G_BYTES + BAR_BYTES;
  static_assert(TOTAL <= 227 * 1024, "k_lora_wgrad shared memory");
};

template <int RB>
__global__ void __launch_bounds__(LORA_WG_THREADS, 1)
    k_lora_wgrad(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1, const LoraWgradParams p) {
  using T = __nv_bfloat16;
  using S = LoraWgradSmem<RB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto sX = [&](int s) { return smem + s * S::X_BYTES; };
  auto sG = [&](int b) { return smem + S::STAGES * S::X_BYTES + b * 2 * S::G_BYTES; };   // [hi, lo]
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + S::STAGES * S::X_BYTES + 4 * S::G_BYTES);
  uint64_t* empty_bar = full_bar + S::STAGES;
  uint64_t* gfull_bar = empty_bar + S::STAGES;   // [2]
  uint64_t* gempty_bar = gfull_bar + 2;          // [2]
  uint64_t* tfull_bar = gempty_bar + 2;          // [2]
  uint64_t* tempty_bar = tfull_bar + 2;          // [2]
  uint64_t* drain_bar = tempty_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr uint32_t ACC_COLS = 2 * RB * 64;
  constexpr uint32_t TCOLS = 2 * ACC_COLS;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&gfull_bar[b], LORA_WG_CONV_WARPS);
      mbar_init(&gempty_bar[b], 1);
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tm0);
    tma_prefetch_desc(&tm1);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();   // dH, and the partial slots' earlier readers
  griddep_launch_dependents();

  const LoraWgradUnits un(p);
  const int64_t u0 = un.first(blockIdx.x), u1 = un.first(blockIdx.x + 1);

  if (warp == 0) {
    // ---------------- TMA producer: 128 columns of the tile a stage ----------------
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool good = true;
    for (int64_t u = u0; good && u < u1; ++u) {
      const int cg = static_cast<int>(u / un.tiles), t = static_cast<int>(u % un.tiles);
      const int side = cg >= un.cg0;
      const int64_t c0 = static_cast<int64_t>(cg - (side ? un.cg0 : 0)) * LORA_WG_COLS;
      const int groups = (p.plan.info(t).y + 15) / 16 * 4;   // whole steps of 16 rows; rows past the count read as zeros
      const int4 r4 = reinterpret_cast<const int4*>(p.plan.rows(t))[lane];
      for (int g = 0; g < 2 && c0 + g * 128 < (side ? p.cols[1] : p.cols[0]); ++g) {
        if (lane == 0) {
          good = mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag);
          if (good) mbar_arrive_expect_tx(&full_bar[stage], static_cast<uint32_t>(2 * groups * 512));
        }
        good = __shfl_sync(0xffffffffu, good, 0);
        if (!good) break;
        if (lane < groups) {
          const int c = static_cast<int>(c0) + g * 128;
          tma_gather4(sX(stage) + lane * 512, side ? &tm1 : &tm0, &full_bar[stage], c, r4);
          tma_gather4(sX(stage) + LORA_TILE * 128 + lane * 512, side ? &tm1 : &tm0, &full_bar[stage], c + 64, r4);
        }
        issued |= 1u << stage;
        if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    if (!good && lane == 0) drain_ring(full_bar, S::STAGES, stage, phase, issued);
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- MMA issuer ----------------
      constexpr uint32_t idesc = idesc_f16(128, RB * 64, true) | IDESC_A_MN | IDESC_B_MN;
      int stage = 0, gb = 0, acc = 0;
      uint32_t phase = 0, g_phase = 0, acc_phase = 0;
      bool good = true, open = false;
      for (int64_t u = u0; good && u < u1; ++u) {
        const int cg = static_cast<int>(u / un.tiles), t = static_cast<int>(u % un.tiles);
        const int side = cg >= un.cg0;
        const int64_t c0 = static_cast<int64_t>(cg - (side ? un.cg0 : 0)) * LORA_WG_COLS;
        const int2 info = p.plan.info(t);
        const int ksteps = (info.y + 15) / 16;
        if (!open && !mbar_wait(&tempty_bar[acc], acc_phase ^ 1u, abort_flag)) break;
        if (!mbar_wait(&gfull_bar[gb], g_phase, abort_flag)) break;
        const uint32_t gs = smem_u32(sG(gb));
        for (int g = 0; g < 2 && c0 + g * 128 < (side ? p.cols[1] : p.cols[0]); ++g) {
          if (!mbar_wait(&full_bar[stage], phase, abort_flag)) { good = false; break; }
          tc_fence_after();
          const uint32_t d = tmem_base + static_cast<uint32_t>(acc) * ACC_COLS + static_cast<uint32_t>(g * RB * 64);
          const uint64_t adesc = sdesc_mn128(smem_u32(sX(stage)), LORA_TILE * 128);
          for (int part = 0; part < 2; ++part) {
            const uint64_t bdesc = sdesc_mn128(gs + part * S::G_BYTES, LORA_TILE * 128);
            for (int k = 0; k < ksteps; ++k)
              umma<2>(d, adesc + 128u * k, bdesc + 128u * k, idesc, (open || (part | k) != 0) ? 1u : 0u);
          }
          umma_commit(&empty_bar[stage]);
          if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!good) break;
        umma_commit(&gempty_bar[gb]);
        if (++gb == 2) { gb = 0; g_phase ^= 1u; }
        open = u + 1 < u1 && t + 1 < p.plan.tile0()[info.x + 1];
        if (!open) {
          umma_commit(&tfull_bar[acc]);
          if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
      }
      drain_mma(drain_bar);
    }
  } else if (warp < 6) {
    // ---------------- epilogue, once per segment ----------------
    const int q = warp & 3;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int64_t u = u0; u < u1;) {
      const int cg = static_cast<int>(u / un.tiles), t = static_cast<int>(u % un.tiles);
      const int side = cg >= un.cg0;
      const int64_t c0 = static_cast<int64_t>(cg - (side ? un.cg0 : 0)) * LORA_WG_COLS;
      const int a = p.plan.info(t).x;
      const int64_t seg0 = static_cast<int64_t>(cg) * un.tiles + p.plan.tile0()[a];
      const int64_t seg1 = static_cast<int64_t>(cg) * un.tiles + p.plan.tile0()[a + 1];
      const int64_t C = (side ? p.cols[1] : p.cols[0]);
      if (!mbar_wait(&tfull_bar[acc], acc_phase, abort_flag)) break;
      tc_fence_after();
      const bool whole = seg0 >= u0 && seg1 <= u1;
      const float s = side ? __ldg(p.scale + a) : 1.0f;
      float* part = p.part + (static_cast<int64_t>(blockIdx.x) * 2 + (seg0 >= u0 ? 1 : 0)) * p.R * LORA_WG_COLS;
      for (int g = 0; g < 2 && c0 + g * 128 < C; ++g) {
        const int64_t col = c0 + g * 128 + q * 32 + lane;
        const uint32_t at = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc) * ACC_COLS + static_cast<uint32_t>(g * RB * 64);
        for (int c = 0; c < p.R; c += 16) {
          uint32_t v[16];
          __syncwarp();
          tmem_ld16(at + static_cast<uint32_t>(c), v);
          tmem_wait16(v);
#pragma unroll
          for (int h = 0; h < 16; h += 8) {
            if (c + h < p.R && col < C) {
              if (!whole) {
#pragma unroll
                for (int i = 0; i < 8; ++i) part[(c + h + i) * LORA_WG_COLS + g * 128 + q * 32 + lane] = __uint_as_float(v[h + i]);
              } else if (side == 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) p.out[0][(static_cast<int64_t>(a) * p.R + c + h + i) * C + col] = from_f<T>(__uint_as_float(v[h + i]));
              } else {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[h + i]) * s;
                *reinterpret_cast<uint4*>(p.out[1] + (static_cast<int64_t>(a) * C + col) * p.R + c + h) =
                    make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty_bar[acc]);
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      u = seg1 < u1 ? seg1 : u1;
    }
  } else {
    // ---------------- G's parts, one tile a unit ----------------
    const int ct = threadIdx.x - 32 * 6;
    constexpr int CH = RB * 8;                                          // 8-value chunks of a row
    constexpr int PER = LORA_TILE * CH / (32 * LORA_WG_CONV_WARPS);    // chunks of a thread
    int gb = 0;
    uint32_t g_phase = 0;
    for (int64_t u = u0; u < u1; ++u) {
      const int cg = static_cast<int>(u / un.tiles), t = static_cast<int>(u % un.tiles);
      const float* G = cg >= un.cg0 ? p.G[1] : p.G[0];
      const int n = p.plan.info(t).y, n16 = (n + 15) / 16 * 16;
      const int* rows = p.plan.rows(t);
      float4 x[PER][2];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = i * 32 * LORA_WG_CONV_WARPS + ct, r = e / CH, c = e % CH;
        x[i][0] = x[i][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < n && 8 * c < p.R) {
          const float4* src = reinterpret_cast<const float4*>(G + static_cast<int64_t>(rows[r]) * p.R + 8 * c);
          x[i][0] = src[0];
          x[i][1] = src[1];
        }
      }
      if (!mbar_wait(&gempty_bar[gb], g_phase ^ 1u, abort_flag)) break;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = i * 32 * LORA_WG_CONV_WARPS + ct, r = e / CH, c = e % CH;
        if (r < n16) {
          const float f[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w, x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
          uint4 hi, lo;
          split8<T>(f, hi, lo);
          uint8_t* d = sG(gb) + (c >> 3) * (LORA_TILE * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
          *reinterpret_cast<uint4*>(d) = hi;
          *reinterpret_cast<uint4*>(d + S::G_BYTES) = lo;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&gfull_bar[gb]);
      if (++gb == 2) { gb = 0; g_phase ^= 1u; }
    }
  }
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, TCOLS);
  }
}

// The segments k_lora_wgrad cut between CTAs, added in CTA order, and zeros
// for adapters without rows. One item is 8 values of R of 256 columns.
__global__ void __launch_bounds__(LORA_WG_COLS) k_lora_wgrad_join(const LoraWgradParams p) {
  using T = __nv_bfloat16;
  griddep_wait();
  const LoraWgradUnits un(p);
  const int rg = p.R / 8;
  const int64_t items = static_cast<int64_t>(un.cgs) * p.plan.L * rg;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int r0 = static_cast<int>(it % rg) * 8;
    const int a = static_cast<int>(it / rg % p.plan.L), cg = static_cast<int>(it / rg / p.plan.L);
    const int side = cg >= un.cg0;
    const int64_t C = (side ? p.cols[1] : p.cols[0]), col = static_cast<int64_t>(cg - (side ? un.cg0 : 0)) * LORA_WG_COLS + threadIdx.x;
    int t0 = 0, t1 = 0;
    if (un.tiles > 0) {
      t0 = p.plan.tile0()[a];
      t1 = p.plan.tile0()[a + 1];
    }
    float f[8] = {};
    if (t0 < t1) {
      const int64_t s0 = static_cast<int64_t>(cg) * un.tiles + t0, s1 = static_cast<int64_t>(cg) * un.tiles + t1;
      const int c0 = un.owner(s0), c1 = un.owner(s1 - 1);
      if (c0 == c1) continue;   // one CTA had it whole
      if (col < C) {
        for (int c = c0; c <= c1; ++c) {
          const float* part = p.part + (static_cast<int64_t>(c) * 2 + (un.first(c) <= s0 ? 1 : 0)) * p.R * LORA_WG_COLS;
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] += part[(r0 + i) * LORA_WG_COLS + threadIdx.x];
        }
      }
    }
    if (col >= C) continue;
    if (side == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p.out[0][(static_cast<int64_t>(a) * p.R + r0 + i) * C + col] = from_f<T>(f[i]);
    } else {
      const float s = __ldg(p.scale + a);
      *reinterpret_cast<uint4*>(p.out[1] + (static_cast<int64_t>(a) * C + col) * p.R + r0) =
          make_uint4(pack2<T>(t0 < t1 ? f[0] * s : 0.0f, t0 < t1 ? f[1] * s : 0.0f), pack2<T>(t0 < t1 ? f[2] * s : 0.0f, t0 < t1 ? f[3] * s : 0.0f),
                     pack2<T>(t0 < t1 ? f[4] * s : 0.0f, t0 < t1 ? f[5] * s : 0.0f), pack2<T>(t0 < t1 ? f[6] * s : 0.0f, t0 < t1 ? f[7] * s : 0.0f));
    }
  }
}

}  // namespace qlin
