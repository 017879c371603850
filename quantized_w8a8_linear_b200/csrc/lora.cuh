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
// rows, and gathers them with 16-byte cp.async copies into the swizzled
// layout the tensor core reads (TMA row gathers, tile::gather4, moved 512
// bytes in about 60 cycles per SM: 54 us against 21 us of HBM time for the
// first product of 16640 x 4096 rows). The products are thin (R <= 128), so
// all three kernels are bound by the 16-bit matrices they read and write, not
// by the tensor cores:
//   k_lora_shrink  H or dH: contraction over K or N;
//   k_lora_expand  Y or dX: contraction over R;
//   k_lora_wgrad   dA and dB: contraction over the rows of an adapter.
// A few rows (a decode step) go through k_lora_rows instead, one launch for
// both products of up to eight rows of one adapter.
//
// H and dH enter the other products as three 16-bit parts, T(h), T of what that
// leaves and T of what both leave, three MMAs on one staged operand: fp32's 24
// bits, so that a row comes out the same as where H stays fp32 (k_lora_rows).
// With two parts, 16 bits in bf16, 2^-17 of the update showed in Y where it
// cancels, and more of Y's elements than an fp32 product has rounded the other
// way; the third one costs the forward pass up to 4% (16640 x 4096 -> 12288,
// rank 64: 197 us in all, 189 with two) and the backward pass 2 to 8%, 17% above
// rank 64. The smallest go first, while the accumulator is small. fp16
// parts are taken of h 2^14 / 2^e with 2^e the largest power of two in the row
// (exact): nothing overflows, all 24 bits of what is above 2^-15 of the row's
// largest are kept, and of the rest all above 2^-39 of it.
//
// All mbarrier waits are bounded (common.cuh).
#pragma once
#include "common.cuh"
#include "vec.cuh"

namespace qlin {

constexpr int LORA_TILE = 128;       // rows of a tile
constexpr int LORA_BK = 64;          // 16-bit elements of a 128-byte swizzled row
constexpr int LORA_MAX_R = 128;
constexpr int LORA_MAX_L = 1024;

// ---------------------------------------------------------------------------
// plan: int32 words
//   [0] M  [1] L  [2] tiles  [3] octets  [4..15] 0
//   tile0 [L + 1]       first tile of each adapter (tile0[L] = tiles)
//   info  [Tmax][2]     adapter and row count of a tile
//   rows  [Tmax][128]   row numbers, in row order; M past the count
//   octet [Omax][12]    adapter, row count, 0, 0, eight row numbers (M past the
//                       count): the rows again in eights, up to LORA_OCTET_M rows
// Tmax = M / 128 + min(L, M) bounds the sum of ceil(rows / 128) over adapters,
// Omax = M / 8 + min(L, M) that of ceil(rows / 8).
// ---------------------------------------------------------------------------
constexpr int LORA_OCTET_M = 256, LORA_OCTET_WORDS = 12;
__host__ __device__ inline int64_t lora_max_tiles(int64_t M, int64_t L) { return M / LORA_TILE + (L < M ? L : M); }
__host__ __device__ inline int64_t lora_max_octets(int64_t M, int64_t L) { return M <= LORA_OCTET_M ? M / 8 + (L < M ? L : M) : 0; }
__host__ __device__ inline int64_t lora_info_at(int64_t L) { return 16 + (L + 4) / 4 * 4; }
__host__ __device__ inline int64_t lora_rows_at(int64_t M, int64_t L) { return lora_info_at(L) + (2 * lora_max_tiles(M, L) + 3) / 4 * 4; }
__host__ __device__ inline int64_t lora_octets_at(int64_t M, int64_t L) { return lora_rows_at(M, L) + LORA_TILE * lora_max_tiles(M, L); }
__host__ __device__ inline int64_t lora_plan_words(int64_t M, int64_t L) { return lora_octets_at(M, L) + LORA_OCTET_WORDS * lora_max_octets(M, L); }

struct LoraPlan {
  const int* w;
  int64_t M, L;
  __device__ __forceinline__ const int* tile0() const { return w + 16; }
  __device__ __forceinline__ int2 info(int t) const { return *reinterpret_cast<const int2*>(w + lora_info_at(L) + 2 * static_cast<int64_t>(t)); }
  __device__ __forceinline__ const int* rows(int t) const { return w + lora_rows_at(M, L) + static_cast<int64_t>(LORA_TILE) * t; }
  __device__ __forceinline__ const int* octet(int o) const { return w + lora_octets_at(M, L) + static_cast<int64_t>(LORA_OCTET_WORDS) * o; }
  // Tiles (octets) of the plan; 0, with QLIN_ERR_INVALID_ARG in the status word, when
  // the buffer holds another problem's plan (its row numbers are not used).
  __device__ __forceinline__ int tiles(bool octets = false) const {
    const int4 h = *reinterpret_cast<const int4*>(w);
    if (h.x == static_cast<int>(M) && h.y == static_cast<int>(L) && h.z >= 0 && h.z <= lora_max_tiles(M, L) && h.w >= 0 && h.w <= lora_max_octets(M, L))
      return octets ? h.w : h.z;
    atomicExch(&g_status, 1 /* QLIN_ERR_INVALID_ARG */);
    return 0;
  }
};

constexpr int LORA_PLAN_THREADS = 1024;

// Stable counting sort of the rows by adapter, in one CTA: warp w counts the
// adapters of its contiguous share of the rows, a scan over (adapter, warp)
// turns the counts into places, and the warps walk their shares again, each
// row's place within 32 rows from the ballot of its equals. No atomics, so
// the order (and every sum over it) is the same in every run. 64 rows take
// 7 us, 16640 rows 16: once a batch, beside two launches for each projection.
__global__ void __launch_bounds__(LORA_PLAN_THREADS) k_lora_plan(const int* idx, int64_t M, int64_t L64, int* plan) {
  extern __shared__ int lora_count[];   // [32][L], then [L] first octets
  __shared__ int warp_total[32], warp_octets[32];
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
  // the adapters of 256 rows from m0 on, eight loads in flight (one by one,
  // 16640 rows took 21 us)
  auto adapters = [&](int64_t m0, int (&a)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t m = m0 + 32 * j + lane;
      a[j] = m < hi ? __ldg(idx + m) : -1;
      if (a[j] >= L) a[j] = -1;
    }
  };
  for (int64_t m0 = lo; m0 < hi; m0 += 256) {
    int as[8];
    adapters(m0, as);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (m0 + 32 * j >= hi) break;
      const int a = as[j];
      const uint32_t same = __match_any_sync(0xffffffffu, a);
      if (a >= 0 && lane == __ffs(same) - 1) mine[a] += __popc(same);
      __syncwarp();
    }
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
  const bool in_octets = M <= LORA_OCTET_M;
  const int octets = in_octets ? (n + 7) / 8 : 0;
  int scan = tiles, oscan = octets;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, scan, o), v = __shfl_up_sync(0xffffffffu, oscan, o);
    if (lane >= o) {
      scan += u;
      oscan += v;
    }
  }
  if (lane == 31) {
    warp_total[warp] = scan;
    warp_octets[warp] = oscan;
  }
  __syncthreads();
  int before = 0, obefore = 0;
  for (int w = 0; w < warp; ++w) {
    before += warp_total[w];
    obefore += warp_octets[w];
  }
  const int first = before + scan - tiles, ofirst = obefore + oscan - octets;
  int* first_octet = lora_count + 32 * L;
  int* octet = plan + lora_octets_at(M, L);
  if (tid < L) {
    tile0[tid] = first;
    if (tid == L - 1) tile0[L] = first + tiles;
    for (int t = 0; t < tiles; ++t) {
      info[2 * (first + t)] = tid;
      info[2 * (first + t) + 1] = n - t * LORA_TILE < LORA_TILE ? n - t * LORA_TILE : LORA_TILE;
    }
    for (int i = n; i < tiles * LORA_TILE; ++i) rows[static_cast<int64_t>(first) * LORA_TILE + i] = static_cast<int>(M);
    for (int w = 0; w < 32; ++w) lora_count[w * L + tid] += first * LORA_TILE;
    first_octet[tid] = ofirst - first * (LORA_TILE / 8);   // of the place lora_count gives a row
    for (int t = 0; t < octets; ++t) {
      int* o = octet + LORA_OCTET_WORDS * (ofirst + t);
      o[0] = tid;
      o[1] = n - 8 * t < 8 ? n - 8 * t : 8;
      o[2] = o[3] = 0;
      for (int i = n - 8 * t; i < 8; ++i) o[4 + i] = static_cast<int>(M);
    }
  }
  if (tid < 16) {
    int total = 0, ototal = 0;
    for (int w = 0; w < 32; ++w) {
      total += warp_total[w];
      ototal += warp_octets[w];
    }
    plan[tid] = tid == 0 ? static_cast<int>(M) : tid == 1 ? L : tid == 2 ? total : tid == 3 ? ototal : 0;
  }
  __syncthreads();
  for (int64_t m0 = lo; m0 < hi; m0 += 256) {
    int as[8];
    adapters(m0, as);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (m0 + 32 * j >= hi) break;
      const int a = as[j], row = static_cast<int>(m0) + 32 * j + lane;
      const uint32_t same = __match_any_sync(0xffffffffu, a);
      const int rank = __popc(same & ((1u << lane) - 1u));
      if (a >= 0) {
        const int at = mine[a] + rank;
        rows[at] = row;
        if (in_octets) octet[LORA_OCTET_WORDS * (first_octet[a] + at / 8) + 4 + at % 8] = row;
      }
      __syncwarp();
      if (a >= 0 && rank == 0) mine[a] += __popc(same);
      __syncwarp();
    }
  }
}

// ---------------------------------------------------------------------------
// helpers
// ---------------------------------------------------------------------------
// Bytes from a matrix's start to its row; rows are below 2^28 and their size below 2^30 bytes, so one multiply-add does.
__device__ __forceinline__ int64_t row_bytes(int row, int bytes) { return static_cast<int64_t>(row) * bytes; }

// 16-byte asynchronous global -> shared copy, or 16 zero bytes (`src` is then not read).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool copy) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(copy ? 16 : 0) : "memory");
}

// Arrives on `bar` once all cp.async copies this thread issued so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// ... or the first `bytes` of them (none, where bytes <= 0) and zeros.
__device__ __forceinline__ void cp_async_upto16(uint32_t dst, const void* src, int64_t bytes) {
  const int n = bytes >= 16 ? 16 : bytes > 0 ? static_cast<int>(bytes) : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(n) : "memory");
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

// 8 fp32 values -> three 16-byte chunks of 16-bit values whose sum is the
// value. Where the first is not finite the others are 0, so an infinite or NaN
// value stays what it is.
template <typename T>
__device__ __forceinline__ void split8(const float (&f)[8], uint4 (&part)[3]) {
  uint16_t h[3][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[0][i] = from_f<T>(f[i]);
    float r = f[i] - to_f<T>(h[0][i]);
    r = fabsf(r) <= fabsf(f[i]) ? r : 0.0f;   // false for NaN and for an infinite first part
    h[1][i] = from_f<T>(r);
    h[2][i] = from_f<T>(r - to_f<T>(h[1][i]));
  }
#pragma unroll
  for (int j = 0; j < 3; ++j)
    part[j] = make_uint4(h[j][0] | (h[j][1] << 16), h[j][2] | (h[j][3] << 16), h[j][4] | (h[j][5] << 16), h[j][6] | (h[j][7] << 16));
}

// The same for 4 values, written to row[0], row[R] and row[2 R] of a split row [3][R].
template <typename T>
__device__ __forceinline__ void store_split4(uint16_t* row, int R, const float4& v) {
  const float f[8] = {v.x, v.y, v.z, v.w};
  uint4 part[3];
  split8<T>(f, part);
#pragma unroll
  for (int j = 0; j < 3; ++j) *reinterpret_cast<uint2*>(row + j * R) = make_uint2(part[j].x, part[j].y);
}

// ---------------------------------------------------------------------------
// k_lora_rows: both products of up to eight rows of one adapter, for batches
// of a few rows. A cluster of eight CTAs takes an octet: each CTA forms H over
// an eighth of K (a warp a row of A, all eight rows of X at once, so A is read
// once), the partial sums meet through distributed shared memory in rank
// order, and each CTA updates an eighth of the columns of Y, a thread a
// column. Latency is all that counts here (64 rows of 32 adapters of rank 16
// move 20 MB, 3 us of HBM time): the CTAs ask for their part of B and Y into
// L2 before they turn to A, and there is no second launch. fp32 FMAs: at these
// sizes the tensor cores would wait for the same bytes. One row 4096 -> 4096
// at rank 16 takes 5 us in a graph of such calls (10 through the two kernels
// below), 64 rows of 32 adapters 7 (21): with A, B and Y in L2. With cold caches
// they take 8 us, and 64 rows of 32 adapters 4096 -> 12288 15 (10 warm).
// ---------------------------------------------------------------------------
constexpr int LORA_ROWS_THREADS = 256, LORA_ROWS_CLUSTER = 8;

struct LoraRowsParams {
  LoraPlan plan;
  int64_t K, N;
  int R;
  const uint16_t* X;    // [M,K]
  const uint16_t* A;    // [L,R,K]
  const uint16_t* B;    // [L,N,R]
  const float* scale;   // [L]
  float* H;             // [M,R], or nullptr: not kept
  uint16_t* Y;          // [M,N]
};

// bytes: the eight rows' part of X (16-bit), partial sums and sums of H
inline int lora_rows_smem(int64_t K, int64_t R) {
  const int64_t kv = (K / 8 + LORA_ROWS_CLUSTER - 1) / LORA_ROWS_CLUSTER;
  return static_cast<int>(8 * kv * 16 + 2 * 8 * R * 4);
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<uint64_t>(p))); }

template <typename T>
__global__ void __launch_bounds__(LORA_ROWS_THREADS, 2) k_lora_rows(const LoraRowsParams p) {
  extern __shared__ uint4 lora_x[];   // [8][kvs] chunks of X, part [8][R], sum [8][R]
  constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank()), R = p.R;
  griddep_wait();
  // the octet's record is asked for beside the plan's header, not after it: the
  // grid ends where the plan's room for octets does
  const int o = blockIdx.x / LORA_ROWS_CLUSTER;
  const int4* record = reinterpret_cast<const int4*>(p.plan.octet(o));
  const int4 head = record[0], rows0 = record[1], rows1 = record[2];
  if (o >= p.plan.tiles(true)) return;   // all CTAs of the cluster
  const int a = head.x, n = head.y;
  const int rows[8] = {rows0.x, rows0.y, rows0.z, rows0.w, rows1.x, rows1.y, rows1.z, rows1.w};
  const int* oct = p.plan.octet(o);
  const int KV = static_cast<int>(p.K / 8), kvs = (KV + LORA_ROWS_CLUSTER - 1) / LORA_ROWS_CLUSTER;
  const int k0 = KV * rank / LORA_ROWS_CLUSTER, kn = KV * (rank + 1) / LORA_ROWS_CLUSTER - k0;
  const int n0 = static_cast<int>(p.N * rank / LORA_ROWS_CLUSTER), n1 = static_cast<int>(p.N * (rank + 1) / LORA_ROWS_CLUSTER);
  const uint16_t* A = p.A + static_cast<int64_t>(a) * R * p.K + 8 * k0;
  const uint16_t* B = p.B + static_cast<int64_t>(a) * p.N * R;
  float* part = reinterpret_cast<float*>(lora_x + 8 * kvs);
  float* sum = part + 8 * R;

  for (int e = tid; e < n * kn; e += LORA_ROWS_THREADS) {
    const int j = e / kn, c = e % kn;
    cp_async16(&lora_x[j * kvs + c], p.X + oct[4 + j] * p.K + 8 * (k0 + c), true);
  }
  cp_async_commit();
  for (int64_t b = 128 * tid; b < 2 * static_cast<int64_t>(n1 - n0) * R; b += 128 * LORA_ROWS_THREADS)
    prefetch_l2(reinterpret_cast<const uint8_t*>(B + static_cast<int64_t>(n0) * R) + b);
  for (int j = warp; j < n; j += LORA_ROWS_THREADS / 32)
    for (int b = 128 * lane; b < 2 * (n1 - n0); b += 128 * 32) prefetch_l2(reinterpret_cast<const uint8_t*>(p.Y + oct[4 + j] * p.N + n0) + b);
  cp_async_wait<0>();
  __syncthreads();

  // H over this CTA's part of K: rows r, r + 8 of A a warp (r < R; R % 8 == 0, the second one may be absent)
  for (int r = warp; r < R; r += 16) {
    const bool two = r + 8 < R;
    const uint4* a0 = reinterpret_cast<const uint4*>(A + static_cast<int64_t>(r) * p.K);
    const uint4* a1 = reinterpret_cast<const uint4*>(A + static_cast<int64_t>(two ? r + 8 : r) * p.K);
    float h[2][8] = {};
#pragma unroll 2
    for (int c = lane; c < kn; c += 32) {
      const uint4 v0 = ld_nc_v4(a0 + c), v1 = ld_nc_v4(a1 + c);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < n) {
          const uint4 x = lora_x[j * kvs + c];
          h[0][j] = fma2_mixed<bf>(x.w, v0.w, fma2_mixed<bf>(x.z, v0.z, fma2_mixed<bf>(x.y, v0.y, fma2_mixed<bf>(x.x, v0.x, h[0][j]))));
          h[1][j] = fma2_mixed<bf>(x.w, v1.w, fma2_mixed<bf>(x.z, v1.z, fma2_mixed<bf>(x.y, v1.y, fma2_mixed<bf>(x.x, v1.x, h[1][j]))));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = warp_sum(h[i][j]);
        if (lane == 0 && (i == 0 || two)) part[j * R + r + 8 * i] = t;
      }
  }
  cluster_sync();
  for (int e = 4 * tid; e < 8 * R; e += 4 * LORA_ROWS_THREADS) {
    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k = 0; k < LORA_ROWS_CLUSTER; ++k) {
      const float4 f = ld_cluster_f4(smem_u32(part + e), static_cast<uint32_t>(k));
      t = make_float4(t.x + f.x, t.y + f.y, t.z + f.z, t.w + f.w);
    }
    *reinterpret_cast<float4*>(sum + e) = t;
    const int j = e / R;
    if (rank == 0 && j < n && p.H != nullptr) *reinterpret_cast<float4*>(p.H + static_cast<int64_t>(oct[4 + j]) * R + e % R) = t;
  }
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");   // this CTA has read its peers' partial sums
  __syncthreads();
  const float s = __ldg(p.scale + a);
  uint16_t* yr[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) yr[j] = p.Y + (j < n ? rows[j] * p.N : 0);
  for (int col = n0 + tid; col < n1; col += 2 * LORA_ROWS_THREADS) {   // columns col and col + 256
    const bool two = col + LORA_ROWS_THREADS < n1;
    const int next = two ? col + LORA_ROWS_THREADS : col;
    uint16_t y0[8], y1[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j < n) {
        y0[j] = yr[j][col];
        y1[j] = yr[j][next];
      }
    }
    float d0[8] = {}, d1[8] = {};
    const uint4* b0 = reinterpret_cast<const uint4*>(B + static_cast<int64_t>(col) * R);
    const uint4* b1 = reinterpret_cast<const uint4*>(B + static_cast<int64_t>(next) * R);
    for (int c = 0; c < R / 8; ++c) {
      float f[8], g[8];
      widen8<T>(__ldg(b0 + c), f);
      widen8<T>(__ldg(b1 + c), g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < n) {
          const float4 u = *reinterpret_cast<const float4*>(sum + j * R + 8 * c), v = *reinterpret_cast<const float4*>(sum + j * R + 8 * c + 4);
          d0[j] = fmaf(f[3], u.w, fmaf(f[2], u.z, fmaf(f[1], u.y, fmaf(f[0], u.x, d0[j]))));
          d1[j] = fmaf(g[3], u.w, fmaf(g[2], u.z, fmaf(g[1], u.y, fmaf(g[0], u.x, d1[j]))));
          d0[j] = fmaf(f[7], v.w, fmaf(f[6], v.z, fmaf(f[5], v.y, fmaf(f[4], v.x, d0[j]))));
          d1[j] = fmaf(g[7], v.w, fmaf(g[6], v.z, fmaf(g[5], v.y, fmaf(g[4], v.x, d1[j]))));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j < n) {
        yr[j][col] = from_f<T>(fmaf(d0[j], s, to_f<T>(y0[j])));
        if (two) yr[j][next] = from_f<T>(fmaf(d1[j], s, to_f<T>(y1[j])));
      }
    }
  }
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");     // no CTA leaves while another reads its partial sums
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
// In the backward pass (W_MN 1) it also leaves dH and the forward's H as split
// rows [3][R] for k_lora_wgrad, whose every CTA reads all of them.
// ---------------------------------------------------------------------------
constexpr int LORA_SHRINK_THREADS = 160;   // warps 0-3 copies, then the epilogue; warp 4 MMA
constexpr int LORA_SHRINK_BK = 128;        // contraction of a stage: 256 bytes of a row

struct LoraShrinkParams {
  LoraPlan plan;
  int64_t C;            // contraction length (K, or N)
  int R;
  const uint16_t* X;    // [M,C]
  const float* scale;   // [L], or nullptr: 1
  float* H;             // [M,R]
  // W_MN 1:
  uint16_t* Hs;         // [M,3,R] the parts of H
  const float* G;       // [M,R] another matrix to split
  uint16_t* Gs;         // [M,3,R]
};

// RB: ceil(R / 64). DEEP: one CTA an SM with four stages, where the tiles would
// not give each SM two of two stages; launch_lora_shrink has the rule and both
// sides' times. Above rank 64 a stage is larger: three of them, one CTA.
// ACCS accumulators take the stages in turn, as many as the CTAs of an SM have
// TMEM for: an MMA cuts its fp32 sum off instead of rounding it, so a sum of
// 4096 products in one chain of 256 MMAs came out 4e-6 of its size too small
// (2.5e-5 where all are positive). Eight chains of 32, added with rounding by
// the epilogue: 4e-7 (torch's fp32 product: 6e-7), at no measurable time.
template <int RB, bool DEEP>
struct LoraShrinkSmem {
  static constexpr int STAGES = RB == 2 ? 3 : DEEP ? 4 : 2;
  static constexpr int ACC_COLS = RB * 64;
  static constexpr int ACCS = (RB == 2 || DEEP ? 512 : 256) / ACC_COLS;
  static constexpr int A_BYTES = 2 * LORA_TILE * 128;   // two halves of 64 columns
  static constexpr int W_BYTES = 2 * RB * 64 * 128;
  static constexpr int STAGE_BYTES = A_BYTES + W_BYTES;
  static constexpr int BAR_BYTES = 8 * (2 * STAGES + 2) + 16;
  static constexpr int TOTAL = 1024 + STAGES * STAGE_BYTES + BAR_BYTES;
  // the partial tile takes the stages' place after the last MMA
  static_assert(LORA_TILE * (RB * 64 + 4) * 4 <= STAGES * STAGE_BYTES, "partial tile");
};

template <typename T, int RB, bool W_MN, bool DEEP>
__global__ void __launch_bounds__(LORA_SHRINK_THREADS)
    k_lora_shrink(const __grid_constant__ CUtensorMap tmW, const LoraShrinkParams p, const int cluster) {
  using S = LoraShrinkSmem<RB, DEEP>;
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
  constexpr uint32_t TCOLS = S::ACCS * S::ACC_COLS;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(&full_bar[s], 129);   // the copying threads, and the copy of W
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(tfull_bar, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmW);
  }
  if (warp == 4) {
    tmem_alloc(tmem_slot, TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // X, the plan and H's earlier readers belong to kernels before this one. In
  // this order: k_lora_expand starts on the release and reads the plan and Y
  // before its own wait, so all that wrote them must have ended by now
  griddep_wait();
  griddep_launch_dependents();

  const int tile = blockIdx.x / cluster;
  const int rank = cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
  // the tile's record and rows are asked for beside the plan's header, not
  // after it: the grid ends where the plan's room for tiles does
  const int* rows = p.plan.rows(tile);
  const int2 info = p.plan.info(tile);
  int src[16];   // a copying thread's rows: r0, r0 + 8, ...; M past the count
#pragma unroll
  for (int i = 0; i < 16; ++i) src[i] = warp < 4 ? rows[(threadIdx.x >> 4) + 8 * i] : 0;
  const bool work = tile < p.plan.tiles();   // the same in all CTAs of the cluster
  const int a = info.x, n = work ? info.y : 0;
  const int kbs = static_cast<int>((p.C + LORA_SHRINK_BK - 1) / LORA_SHRINK_BK);
  const int kb0 = static_cast<int>(static_cast<int64_t>(kbs) * rank / cluster);
  const int kb1 = static_cast<int>(static_cast<int64_t>(kbs) * (rank + 1) / cluster);
  const int Rp = (p.R + 15) / 16 * 16;

  if (work && warp < 4) {
    // ---------------- copies: chunk c of rows r0, r0 + 8, ..., 16 lanes a row ----------------
    const int c = lane & 15, r0 = threadIdx.x >> 4;
    const int C = static_cast<int>(p.C), M = static_cast<int>(p.plan.M);
    const uint32_t off = static_cast<uint32_t>((c >> 3) * (LORA_TILE * 128) + r0 * 128 + (((c & 7) ^ r0) << 4));
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool good = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      good = mbar_wait_warp(&empty_bar[stage], phase ^ 1u, abort_flag);
      if (!good) break;
      if (threadIdx.x == 0) {
        mbar_arrive_expect_tx(&full_bar[stage], static_cast<uint32_t>(W_MN ? S::W_BYTES : 2 * Rp * 128));
        if constexpr (W_MN) {
#pragma unroll
          for (int b = 0; b < RB; ++b) tma_load_3d(sW(stage) + b * 16384, &tmW, &full_bar[stage], b * 64, kb * LORA_SHRINK_BK, a);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) tma_load_3d(sW(stage) + h * RB * 8192, &tmW, &full_bar[stage], kb * LORA_SHRINK_BK + h * 64, 0, a);
        }
      }
      const uint32_t d = smem_u32(sA(stage)) + off;
      const bool in = kb * LORA_SHRINK_BK + 8 * c < C;
      const uint8_t* x = reinterpret_cast<const uint8_t*>(p.X + kb * LORA_SHRINK_BK + 8 * c);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (src[i] < M) cp_async16_or_zero(d + 1024u * i, x + row_bytes(src[i], 2 * C), in);
      cp_async_arrive(&full_bar[stage]);
      issued |= 1u << stage;
      if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
    }
    cp_async_commit();
    cp_async_wait<0>();
    // ---------------- epilogue: row q * 32 + lane of the tile ----------------
    const int q = warp;
    const int r = q * 32 + lane;
    good = good && mbar_wait_warp(tfull_bar, 0, abort_flag);
    if (!good && threadIdx.x == 0) drain_ring(full_bar, S::STAGES, stage, phase, issued);   // else the MMAs have read them all
    __syncwarp();
    good = good && kb1 > kb0;
    tc_fence_after();
    const float s = p.scale != nullptr ? __ldg(p.scale + a) : 1.0f;
    float* out = cluster > 1 ? reinterpret_cast<float*>(smem) + r * (Rp + 4) : p.H + static_cast<int64_t>(r < n ? rows[r] : 0) * p.R;
    if (q * 32 < n) {
      const int accs = kb1 - kb0 < S::ACCS ? kb1 - kb0 : S::ACCS;   // those with a sum
      for (int c0 = 0; c0 < p.R; c0 += 16) {
        float sum[16] = {};
#pragma unroll
        for (int b0 = 0; b0 < S::ACCS; b0 += 4) {
          uint32_t v[4][16];
          __syncwarp();
#pragma unroll
          for (int b = 0; b < 4; ++b) tmem_ld16(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>((b0 + b) * S::ACC_COLS + c0), v[b]);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            tmem_wait16(v[b]);
            if (b0 + b < accs) {
#pragma unroll
              for (int i = 0; i < 16; ++i) sum[i] += __uint_as_float(v[b][i]);
            }
          }
        }
        if (r < n) {
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            if (c0 + i < p.R) {
              float4 f = make_float4(sum[i], sum[i + 1], sum[i + 2], sum[i + 3]);
              if (!good) f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              if (cluster == 1) {
                f = make_float4(f.x * s, f.y * s, f.z * s, f.w * s);
                if constexpr (W_MN) store_split4<T>(p.Hs + static_cast<int64_t>(rows[r]) * 3 * p.R + c0 + i, p.R, f);
              }
              *reinterpret_cast<float4*>(out + c0 + i) = f;
            }
          }
        }
      }
    }
    tc_fence_before();
  } else if (work && lane == 0) {
    // ---------------- MMA issuer ----------------
    bool good = injected_wait(drain_bar, abort_flag);
    constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
    const uint32_t idesc = W_MN ? (idesc_f16(LORA_TILE, RB * 64, bf) | IDESC_B_MN) : idesc_f16(LORA_TILE, Rp, bf);
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; good && kb < kb1; ++kb) {
      good = mbar_wait(&full_bar[stage], phase, abort_flag);
      if (!good) break;
      fence_proxy_async_smem();   // X was written by cp.async, through the generic proxy
      tc_fence_after();
      const uint32_t as = smem_u32(sA(stage)), ws = smem_u32(sW(stage));
      const uint32_t d = tmem_base + static_cast<uint32_t>((kb - kb0) % S::ACCS * S::ACC_COLS);
#pragma unroll
      for (int k = 0; k < LORA_SHRINK_BK / 16; ++k) {
        const uint64_t adesc = sdesc_k128(as + (k >> 2) * (LORA_TILE * 128)) + 2u * (k & 3);
        const uint64_t bdesc = W_MN ? sdesc_mn128(ws, 16384u) + 128u * k : sdesc_k128(ws + (k >> 2) * (RB * 8192)) + 2u * (k & 3);
        umma<2>(d, adesc, bdesc, idesc, (kb - kb0 >= S::ACCS || k != 0) ? 1u : 0u);
      }
      umma_commit(&empty_bar[stage]);
      if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
    }
    if (good) umma_commit(tfull_bar);
    drain_mma(drain_bar);
  }
  // TMEM goes back before the CTAs of a cluster wait for one another: a peer
  // may be waiting for another kernel's on its SM
  __syncthreads();
  if (warp == 4) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, TCOLS);
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
        sum = make_float4(sum.x * s, sum.y * s, sum.z * s, sum.w * s);
        const int64_t row = p.plan.rows(tile)[r];
        *reinterpret_cast<float4*>(p.H + row * p.R + c) = sum;
        if constexpr (W_MN) store_split4<T>(p.Hs + row * 3 * p.R + c, p.R, sum);
      }
    }
    cluster_sync();   // no CTA leaves while another reads its partial tile
  }
  if constexpr (W_MN) {
    const int r4 = p.R / 4, mine = rank < n ? (n - rank + cluster - 1) / cluster : 0;
    for (int e = threadIdx.x; e < mine * r4; e += LORA_SHRINK_THREADS) {
      const int64_t row = p.plan.rows(tile)[rank + e / r4 * cluster];
      const int c = e % r4 * 4;
      store_split4<T>(p.Gs + row * 3 * p.R + c, p.R, *reinterpret_cast<const float4*>(p.G + row * p.R + c));
    }
  }
}

// ---------------------------------------------------------------------------
// k_lora_expand: Y[rows of the tile] += s H V^T, 128 columns a unit, H in parts.
//   V_MN 0: V = B[a] [N, R], K-major;   1: V = A[a] [R, K] read as its
//   transpose, MN-major, with Y = dX and K columns.
// Persistent, one CTA an SM: the units (tile, 128 columns), columns fastest,
// are cut into one equal range per CTA, so that every SM moves the same number
// of bytes whatever the tiles; a range spans few tiles, whose H is split into
// its parts once each. Y comes in by cp.async, up to three units ahead, into
// rows of 272 bytes (a row a thread and a row a few lanes are both free of
// bank conflicts), is updated there by the thread that holds the row's
// accumulator, and leaves in 128-byte pieces of rows; two groups of eight
// warps take turns at the units, since one group's chain of waits, loads and
// stores took longer than a unit's bytes. 256 bytes of a row at a
// time are what HBM wants: reading and writing 128 rows of 24 KB in place,
// walked in pieces of 64, 128, 256 and 512 bytes, runs at 4.2, 4.6, 5.2 and
// 5.3 TB/s; 16640 rows of 12288 at rank 64 take 151 us, 5.4 TB/s. The copies
// of Y and V start before the kernel that makes H has ended (programmatic
// dependent launch); only the readers of H wait for it.
//   VEC false: rows of Y that are not multiples of 16 bytes. A row's piece
// then lies `shift` bytes into its 17 aligned 16-byte chunks, in shared memory
// as in global memory, so that the copies in stay whole chunks; on the way out
// the two chunks that a piece shares with its neighbours go element by element.
// ---------------------------------------------------------------------------
constexpr int LORA_EXPAND_THREADS = 704;   // warps 0-3 copy Y, warp 4 copies V, warp 5 MMA, warps 6-21 split H and the epilogue
constexpr int LORA_EXPAND_BN = 128;

struct LoraExpandParams {
  LoraPlan plan;
  int64_t N;            // columns of Y
  int R;
  const float* scale;   // [L], or nullptr: 1
  const float* H;       // [M,R]
  uint16_t* Y;          // [M,N]
};

template <int RB>
struct LoraExpandSmem {
  static constexpr int V_STAGES = RB == 1 ? 2 : 3;                     // each 64 of R
  static constexpr int Y_STAGES = RB == 1 ? 4 : 2;
  static constexpr int H_BYTES = RB * LORA_TILE * 128;                 // one part
  static constexpr int V_BYTES = LORA_EXPAND_BN * 128;
  static constexpr int Y_ROW = 272;
  static constexpr int Y_BYTES = LORA_TILE * Y_ROW;
  static constexpr int BAR_BYTES = 8 * (2 * V_STAGES + 2 * Y_STAGES + 7) + 16;
  static constexpr int UP_BYTES = 2 * LORA_TILE * 4;                   // fp16: powers of two of the rows
  static constexpr int TOTAL = 1024 + 3 * H_BYTES + V_STAGES * V_BYTES + Y_STAGES * Y_BYTES + UP_BYTES + BAR_BYTES;
  static_assert(TOTAL <= 227 * 1024, "k_lora_expand shared memory");
};

template <typename T, int RB, bool V_MN, bool VEC>
__global__ void __launch_bounds__(LORA_EXPAND_THREADS, 1) k_lora_expand(const __grid_constant__ CUtensorMap tmV, const LoraExpandParams p) {
  using S = LoraExpandSmem<RB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sH = smem;   // [3 parts][RB][128 rows][128 bytes]
  auto sV = [&](int s) { return smem + 3 * S::H_BYTES + s * S::V_BYTES; };
  auto sY = [&](int s) { return smem + 3 * S::H_BYTES + S::V_STAGES * S::V_BYTES + s * S::Y_BYTES; };
  float* sUp = reinterpret_cast<float*>(smem + 3 * S::H_BYTES + S::V_STAGES * S::V_BYTES + S::Y_STAGES * S::Y_BYTES);   // [2][128]
  uint64_t* vfull_bar = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sUp) + S::UP_BYTES);
  uint64_t* vempty_bar = vfull_bar + S::V_STAGES;
  uint64_t* yfull_bar = vempty_bar + S::V_STAGES;
  uint64_t* yempty_bar = yfull_bar + S::Y_STAGES;
  uint64_t* tfull_bar = yempty_bar + S::Y_STAGES;   // [2]
  uint64_t* tempty_bar = tfull_bar + 2;             // [2]
  uint64_t* hfull_bar = tempty_bar + 2;
  uint64_t* hempty_bar = hfull_bar + 1;
  uint64_t* drain_bar = hempty_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr uint32_t TCOLS = 2 * LORA_EXPAND_BN;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::V_STAGES; ++s) {
      mbar_init(&vfull_bar[s], 1);
      mbar_init(&vempty_bar[s], 1);
    }
    for (int s = 0; s < S::Y_STAGES; ++s) {
      mbar_init(&yfull_bar[s], 128);
      mbar_init(&yempty_bar[s], 8);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], 8);
    }
    mbar_init(hfull_bar, 16);
    mbar_init(hempty_bar, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmV);
  }
  if (warp == 5) {
    tmem_alloc(tmem_slot, TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // The plan, Y and V are read from here on, H only behind griddep_wait: the
  // kernel before this one is k_lora_shrink, k_lora_wgrad or its join, and none
  // of them lets this one start before all earlier kernels have ended
  const int nbs = static_cast<int>((p.N + LORA_EXPAND_BN - 1) / LORA_EXPAND_BN);
  const int64_t units = static_cast<int64_t>(p.plan.tiles()) * nbs;
  const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  const int t0 = static_cast<int>(u0 / nbs), nb0 = static_cast<int>(u0 % nbs);   // first tile and columns
  // byte of its aligned 16-byte chunk at which `row`, and any piece of it, starts (a unit's columns are 256 bytes)
  auto shift_of = [&](int row) { return VEC ? 0 : static_cast<int>((2u * static_cast<uint32_t>(row) * static_cast<uint32_t>(p.N)) & 15u); };

  if (warp < 4) {
    // ---------------- copies of Y: chunk c of rows r0, r0 + 8, ..., 16 lanes a row ----------------
    const int c = lane & 15, r0 = threadIdx.x >> 4;
    const int64_t all = 2 * p.plan.M * p.N;   // bytes of Y
    const int row_size = static_cast<int>(2 * p.N), M = static_cast<int>(p.plan.M);
    const uint8_t* Y = reinterpret_cast<const uint8_t*>(p.Y);
    // a row's first aligned chunk, its shift in the low bits; -1 past the count
    int64_t row_at[16];
    int stage = 0;
    uint32_t phase = 0;
    bool good = true, next = true;
    for (int64_t u = u0, t = t0, nb = nb0; u < u1; ++u) {
      if (next) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int row = p.plan.rows(static_cast<int>(t))[r0 + 8 * i];   // M past the count
          row_at[i] = row < M ? row_bytes(row, row_size) : -1;
        }
      }
      good = mbar_wait_warp(&yempty_bar[stage], phase ^ 1u, abort_flag);
      if (!good) break;
      const int n0 = static_cast<int>(nb) * LORA_EXPAND_BN;
      const uint32_t d = smem_u32(sY(stage)) + r0 * S::Y_ROW + 16 * c;
      if (nb + 2 < nbs) {   // whole units whose chunks end within the row's matrix
        const uint8_t* y = Y + 2 * n0 + 16 * c;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (row_at[i] >= 0) {
            cp_async16_or_zero(d + 8 * S::Y_ROW * i, y + (VEC ? row_at[i] : row_at[i] & ~int64_t{15}), true);
            if (!VEC && c == 0 && (row_at[i] & 15) != 0) cp_async16_or_zero(d + 8 * S::Y_ROW * i + 256, y + 256 + (row_at[i] & ~int64_t{15}), true);
          }
        }
      } else {
        const int bytes = static_cast<int>(2 * (p.N - n0 < LORA_EXPAND_BN ? p.N - n0 : LORA_EXPAND_BN));
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int shift = VEC ? 0 : static_cast<int>(row_at[i] & 15);
          const int64_t at = row_at[i] - shift + 2 * n0 + 16 * c;
          if (row_at[i] >= 0 && 16 * c < shift + bytes) cp_async_upto16(d + 8 * S::Y_ROW * i, Y + at, VEC ? 16 : all - at);
          if (!VEC && row_at[i] >= 0 && c == 0 && 256 < shift + bytes) cp_async_upto16(d + 8 * S::Y_ROW * i + 256, Y + at + 256, all - at - 256);
        }
      }
      cp_async_arrive(&yfull_bar[stage]);
      if (++stage == S::Y_STAGES) { stage = 0; phase ^= 1u; }
      next = ++nb == nbs;
      if (next) {
        nb = 0;
        ++t;
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp == 4) {
    if (lane == 0) {
      // ---------------- TMA producer: V ----------------
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool good = true;
      int a = u0 < u1 ? p.plan.info(t0).x : 0;
      for (int64_t u = u0, t = t0, nb = nb0; u < u1; ++u) {
        const int n0 = static_cast<int>(nb) * LORA_EXPAND_BN;
        for (int b = 0; b < RB; ++b) {   // 64 of R a stage
          good = mbar_wait(&vempty_bar[stage], phase ^ 1u, abort_flag);
          if (!good) break;
          mbar_arrive_expect_tx(&vfull_bar[stage], S::V_BYTES);
          if constexpr (V_MN) {
#pragma unroll
            for (int h = 0; h < 2; ++h) tma_load_3d(sV(stage) + h * 8192, &tmV, &vfull_bar[stage], n0 + 64 * h, b * 64, a);
          } else {
            tma_load_3d(sV(stage), &tmV, &vfull_bar[stage], b * 64, n0, a);
          }
          issued |= 1u << stage;
          if (++stage == S::V_STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!good) break;
        if (++nb == nbs) {
          nb = 0;
          if (u + 1 < u1) a = p.plan.info(static_cast<int>(++t)).x;
        }
      }
      drain_ring(vfull_bar, S::V_STAGES, stage, phase, issued);
    }
  } else if (warp == 5) {
    if (lane == 0) {
      // ---------------- MMA issuer ----------------
      constexpr uint32_t idesc = idesc_f16(LORA_TILE, LORA_EXPAND_BN, std::is_same<T, __nv_bfloat16>::value) | (V_MN ? IDESC_B_MN : 0u);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0, h_phase = 0;
      bool next = true, good = injected_wait(drain_bar, abort_flag);
      for (int64_t u = u0, nb = nb0; good && u < u1; ++u) {
        if (next) {
          if (!mbar_wait(hfull_bar, h_phase, abort_flag)) break;
          h_phase ^= 1u;
        }
        if (!mbar_wait(&tempty_bar[acc], acc_phase ^ 1u, abort_flag)) break;
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * LORA_EXPAND_BN);
        for (int b = 0; b < RB; ++b) {   // 64 of R
          good = mbar_wait(&vfull_bar[stage], phase, abort_flag);
          if (!good) break;
          tc_fence_after();
          const uint32_t v = smem_u32(sV(stage)), h = smem_u32(sH) + static_cast<uint32_t>(b * (LORA_TILE * 128));
#pragma unroll
          for (int k = 0; k < 12; ++k) {   // the smallest part of H first; zeros past R
            const int i = k & 3, part = 2 - (k >> 2);
            const uint64_t adesc = sdesc_k128(h + part * S::H_BYTES) + 2u * i;
            const uint64_t bdesc = V_MN ? sdesc_mn128(v, 8192u) + 128u * i : sdesc_k128(v) + 2u * i;
            umma<2>(d, adesc, bdesc, idesc, k != 0 || b != 0 ? 1u : 0u);
          }
          umma_commit(&vempty_bar[stage]);
          if (++stage == S::V_STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!good) break;
        umma_commit(&tfull_bar[acc]);
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        next = ++nb == nbs;
        if (next) {
          nb = 0;
          umma_commit(hempty_bar);
        }
      }
      drain_mma(drain_bar);
    }
  } else {
    // ---------------- H's parts, then the epilogue: rows 32 q .. 32 q + 31, columns 64 half .. 64 half + 63 ----------------
    const int q = warp & 3, half = (warp - 6) >> 2 & 1, group = warp >= 14;   // group: of the units it takes, and of their accumulators
    const uint32_t tmem = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(group * LORA_EXPAND_BN + 64 * half);
    int stage = 0, n = 0, my_row = 0;
    float s = 1.0f;    // scale[a], times the power of two of the lane's row (fp16)
    uint32_t phase = 0, acc_phase = 0, h_phase = 0;
    int up_at = 0;     // half of sUp: tiles alternate, since a warp may be splitting the next one while another has not read this one's
    bool next = true, good = true;
    for (int64_t u = u0, t = t0, nb = nb0; u < u1; ++u) {
      if (next) {
        const int2 info = p.plan.info(static_cast<int>(t));
        const int at = p.plan.rows(static_cast<int>(t))[q * 32 + lane];
        n = info.y - q * 32;
        my_row = n > lane ? at : 0;
        if (u == u0) {
          griddep_wait();    // H
        } else {             // the MMAs that read the previous tile's parts
          good = mbar_wait_warp(hempty_bar, h_phase, abort_flag);
          if (!good) break;
          h_phase ^= 1u;
        }
        s = p.scale != nullptr ? __ldg(p.scale + info.x) : 1.0f;
        constexpr bool F16 = std::is_same<T, __half>::value;
        constexpr int CH = RB * 8;   // 8-value chunks of a row: lanes of a warp that share a row
        // the four warps of these rows take every fourth step of 32 / CH rows
#pragma unroll
        for (int i0 = 0; i0 < CH; i0 += 4) {
          const int e = (i0 + 2 * group + half) * 32 + lane, r = e / CH, c = e % CH;
          const int row = __shfl_sync(0xffffffffu, my_row, r), rr = q * 32 + r;
          float f[8] = {};
          if (r < n && 8 * c < p.R) {
            const float4* src = reinterpret_cast<const float4*>(p.H + static_cast<int64_t>(row) * p.R + 8 * c);
            const float4 x = src[0], y = src[1];
            f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
            f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
          }
          if constexpr (F16) {
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
#pragma unroll
            for (int o = CH / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            // up = 2^(e - 14) with 2^e <= max < 2^(e+1), down = 1 / up; rows with infinities or NaN keep 1
            const uint32_t em = __float_as_uint(m) >> 23, eb = em > 15u ? em - 14u : 1u;
            const float down = em < 255u ? __uint_as_float((254u - eb) << 23) : 1.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= down;
            if (c == 0) sUp[up_at * LORA_TILE + rr] = em < 255u ? __uint_as_float(eb << 23) : 1.0f;
          }
          uint4 part[3];
          split8<T>(f, part);
          uint8_t* h = sH + (c >> 3) * (LORA_TILE * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4);
#pragma unroll
          for (int j = 0; j < 3; ++j) *reinterpret_cast<uint4*>(h + j * S::H_BYTES) = part[j];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(hfull_bar);
        if constexpr (F16) {   // the power of two of the lane's own row, from the warp that split it
          good = mbar_wait_warp(hfull_bar, static_cast<uint32_t>(up_at), abort_flag);
          if (!good) break;
          s *= sUp[up_at * LORA_TILE + q * 32 + lane];
          up_at ^= 1;
        }
      }
      if (((u - u0) & 1) == group) {
      good = mbar_wait_warp(&tfull_bar[group], acc_phase, abort_flag) && mbar_wait_warp(&yfull_bar[stage], phase, abort_flag);
      if (!good) break;
      acc_phase ^= 1u;
      tc_fence_after();
      if (n > 0) {
        const int n0 = static_cast<int>(nb) * LORA_EXPAND_BN;
        uint8_t* yr = sY(stage) + q * 32 * S::Y_ROW;   // the warp's rows
        const int shift = shift_of(my_row);
        // VEC false: the piece from the 8-byte word it starts in; `late`: it starts
        // in that word's second half; `odd`: in the upper 16 bits of a 32-bit word,
        // so that pairs of columns straddle two
        uint8_t* mine = yr + lane * S::Y_ROW + 128 * half + (VEC ? 0 : shift & ~7);
        const bool late = !VEC && (shift & 4) != 0;
        const uint32_t odd = VEC ? 0 : (shift & 2) * 8;
        uint2 carry = make_uint2(0, 0);              // the two words behind the ones done
        uint32_t before = 0, last = 0;               // the previous pair, the word of it not yet written (late)
        if constexpr (!VEC) carry = *reinterpret_cast<const uint2*>(mine);
#pragma unroll
        for (int c = 0; c < 64; c += 16) {
          uint32_t v[16];
          tmem_ld16(tmem + static_cast<uint32_t>(c), v);
          tmem_wait16(v);
          auto sum_of = [&](int j) { return __uint_as_float(v[j]); };
          if constexpr (VEC) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint4* at = reinterpret_cast<uint4*>(mine + 2 * c + 16 * h);
              float f[8];
              widen8<T>(*at, f);
#pragma unroll
              for (int i = 0; i < 8; ++i) f[i] = fmaf(sum_of(8 * h + i), s, f[i]);
              *at = narrow8<T>(f);
            }
          } else {
            // 8-byte accesses: rows 272 bytes apart meet in every eighth lane's
            // banks, so 32-bit ones took four passes each (63% of the LSU's time)
            uint2* at = reinterpret_cast<uint2*>(mine + 2 * c);   // words 0 .. 7, and the next two
            uint32_t w[10] = {carry.x, carry.y};
#pragma unroll
            for (int i = 1; i < 5; ++i) {
              carry = at[i];
              w[2 * i] = carry.x;
              w[2 * i + 1] = carry.y;
            }
            uint32_t sums[8];   // the words of the updated pairs, from word `late` on
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t lo = late ? w[i + 1] : w[i], hi = late ? w[i + 2 < 10 ? i + 2 : 9] : w[i + 1];
              const uint32_t pair = __funnelshift_r(lo, hi, odd);
              const uint32_t sum = narrow2<T>(fmaf(sum_of(2 * i), s, to_f<T>(static_cast<uint16_t>(pair))),
                                              fmaf(sum_of(2 * i + 1), s, to_f<T>(static_cast<uint16_t>(pair >> 16))));
              sums[i] = __funnelshift_l(before, sum, odd);
              before = sum;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint2 two = late ? make_uint2(i == 0 ? last : sums[2 * i - 1], sums[2 * i]) : make_uint2(sums[2 * i], sums[2 * i + 1]);
              if (c > 0 || i > 0) {
                at[i] = two;
              } else {   // the piece's first word: what lies before it is another warp's
                uint32_t* first = reinterpret_cast<uint32_t*>(at) + late;
                if (odd) reinterpret_cast<uint16_t*>(first)[1] = static_cast<uint16_t>(sums[0] >> 16);
                else *first = sums[0];
                if (!late) first[1] = sums[1];
              }
            }
            last = sums[7];
          }
        }
        if constexpr (!VEC) {   // behind the last whole words; what lies after the piece is another warp's
          uint32_t* end = reinterpret_cast<uint32_t*>(mine + 128);
          if (late) *end++ = last;
          if (odd) *reinterpret_cast<uint16_t*>(end) = static_cast<uint16_t>(before >> 16);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty_bar[group]);   // the accumulator is in shared memory
        // out: eight lanes a row, 16-byte chunk c of the warp's 128 bytes of it
        const int c = lane & 7;
        const int N = static_cast<int>(p.N), col = n0 + 64 * half;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i * 4 + (lane >> 3);
          const int row = __shfl_sync(0xffffffffu, my_row, r);
          if (r < n) {
            const uint8_t* src = yr + r * S::Y_ROW + 128 * half;
            uint8_t* dst = reinterpret_cast<uint8_t*>(p.Y + col) + row_bytes(row, 2 * N);
            if constexpr (VEC) {
              if (col + 8 * c < N) *reinterpret_cast<uint4*>(dst + 16 * c) = *reinterpret_cast<const uint4*>(src + 16 * c);
            } else {
              const int sh = shift_of(row);
              const int cols = N - col < 64 ? N - col : 64;
              // with a shift, the piece has `head` elements before its first whole
              // chunk and 8 - head behind its last one: one of the eight for each lane
              const int head = (16 - sh) / 2 & 7, e0 = 8 * c + head;
              auto element = [&](int e) {
                if (e < cols) *reinterpret_cast<uint16_t*>(dst + 2 * e) = *reinterpret_cast<const uint16_t*>(src + sh + 2 * e);
              };
              if (head == 0 || c < 7) {
                if (e0 + 8 <= cols) {
                  *reinterpret_cast<uint4*>(dst + 2 * e0) = *reinterpret_cast<const uint4*>(src + sh + 2 * e0);
                } else {
                  for (int e = e0; e < e0 + 8; ++e) element(e);   // the matrix's last columns
                }
              }
              if (head != 0) element(c < head ? c : 56 + c);
            }
          }
        }
      } else if (lane == 0) {
        mbar_arrive(&tempty_bar[group]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&yempty_bar[stage]);
      }
      if (++stage == S::Y_STAGES) { stage = 0; phase ^= 1u; }
      next = ++nb == nbs;
      if (next) {
        nb = 0;
        ++t;
      }
    }
  }
  __syncthreads();
  griddep_wait();
  if (warp == 5) {
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
// transposed. Sums stay in TMEM over the tiles of an adapter: an MMA cuts its
// accumulator off instead of rounding it, so every LORA_WG_CHAIN tiles the
// epilogue adds it, rounded, to sums of its own beside it (of the bf16 sums over
// 8192 rows of positive products one chain put 0.28% on the wrong side of a
// rounding, chains of 1024 rows 0.012%). The accumulators of a unit's two MMAs
// are handed back one by one, and the copies run on meanwhile: 154 us for a
// backward pass that took 157 with two accumulators in turn. An adapter whose
// tiles are cut between CTAs leaves fp32 partial sums, slot 0 for a CTA's
// first segment if it began before, slot 1 for the last one, and
// k_lora_wgrad_join adds them in CTA order. 8191 rows, 4096 and 12288 columns,
// rank 64: 70 us, 3.8 TB/s of X and dY (the join 9).
// bf16 only: G's parts need fp32's exponent range (a power of two per row, as
// k_lora_expand takes out, does not leave a sum over rows).
// ---------------------------------------------------------------------------
constexpr int LORA_WG_THREADS = 416;   // warps 0-3 copy X, warp 4 MMA, warps 5-8 epilogue, warps 9-12 copy G
constexpr int LORA_WG_COLS = 256;      // columns of a unit: two MMAs of M = 128
constexpr int LORA_WG_ROWS = 64;       // rows of a block of MMAs: a tile has one or two
constexpr int LORA_WG_CHAIN = 8;       // tiles of a chain of MMAs (4 above rank 64)

struct LoraWgradParams {
  LoraPlan plan;
  int R, ctas;
  int64_t cols[2];       // K, N
  const uint16_t* X[2];  // X [M,K], dY [M,N]
  const uint16_t* G[2];  // dH, H as split rows [M,3,R]
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
  // first unit of a CTA (of the CTAs past the last one with units: `units`)
  __device__ __forceinline__ int64_t first(int64_t cta) const { return cta < ctas ? units * cta / ctas : units; }
};

template <int RB>
struct LoraWgradSmem {
  static constexpr int STAGES = 4;
  static constexpr int X_BYTES = 2 * LORA_TILE * 128;            // 128 columns of the tile: two 64-column halves
  static constexpr int G_BUFS = 2;
  static constexpr int G_ROWS = LORA_TILE / RB;                  // rows of a buffer of G: a tile, above rank 64 half of one
  static constexpr int G_BYTES = RB * G_ROWS * 128;              // one part
  static constexpr int BAR_BYTES = 8 * (2 * STAGES + 2 * G_BUFS + 5) + 16;
  static constexpr int TOTAL = 1024 + STAGES * X_BYTES + G_BUFS * 3 * G_BYTES + BAR_BYTES;
  static_assert(TOTAL <= 227 * 1024, "k_lora_wgrad shared memory");
};

template <int RB>
__global__ void __launch_bounds__(LORA_WG_THREADS, 1) k_lora_wgrad(const LoraWgradParams p) {
  using T = __nv_bfloat16;
  using S = LoraWgradSmem<RB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto sX = [&](int s) { return smem + s * S::X_BYTES; };
  auto sG = [&](int b) { return smem + S::STAGES * S::X_BYTES + b * 3 * S::G_BYTES; };   // [3 parts]
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + S::STAGES * S::X_BYTES + S::G_BUFS * 3 * S::G_BYTES);
  uint64_t* empty_bar = full_bar + S::STAGES;
  uint64_t* gfull_bar = empty_bar + S::STAGES;
  uint64_t* gempty_bar = gfull_bar + S::G_BUFS;
  uint64_t* tfull_bar = gempty_bar + S::G_BUFS;           // [2], of the accumulators of a unit's two MMAs
  uint64_t* tempty_bar = tfull_bar + 2;          // [2]
  uint64_t* drain_bar = tempty_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // R <= 64: one MMA multiplies all parts (N = 192: side by side, added by the
  // epilogue), so that X's tile is read from shared memory once; above, one MMA
  // a part, into the same accumulator. A buffer of G then holds 64 rows (four
  // buffers of 32 rows: 8192 x 4096 -> 12288 at rank 72, the whole backward
  // pass, 235 us; two of 64 rows 210).
  constexpr bool ALL = RB == 1;
  constexpr uint32_t G_COLS = ALL ? 192 : 128;   // accumulator columns of 128 columns of X
  constexpr uint32_t SUMS = 2 * G_COLS, SUM_COLS = RB * 64;   // the rounded sums behind the two accumulators
  constexpr uint32_t TCOLS = 512;
  static_assert(SUMS + 2 * SUM_COLS <= TCOLS, "TMEM");
  constexpr int CHAIN = LORA_WG_CHAIN / RB;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(&full_bar[s], 128);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < S::G_BUFS; ++b) {
      mbar_init(&gfull_bar[b], 128);
      mbar_init(&gempty_bar[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 4) {
    tmem_alloc(tmem_slot, TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();   // dH, and the partial slots' earlier readers
  griddep_launch_dependents();   // in this order: k_lora_expand reads the plan and dX before its own wait

  const LoraWgradUnits un(p);
  const int64_t u0 = un.first(blockIdx.x), u1 = un.first(blockIdx.x + 1);

  if (warp < 4) {
    // ---------------- copies: 128 columns of the tile a stage; chunk c of rows r0 .. r0 + 15, 16 lanes a row ----------------
    const int c = lane & 15, r0 = (threadIdx.x >> 4) * 16;
    const uint32_t off = static_cast<uint32_t>((c >> 3) * (LORA_TILE * 128) + r0 * 128);
    int stage = 0;
    uint32_t phase = 0;
    bool good = true;
    int4 ahead[4];   // the next unit's rows
    int ahead_n = 0;
    auto look_ahead = [&](int t) {
      ahead_n = p.plan.info(t).y;
#pragma unroll
      for (int i = 0; i < 4; ++i) ahead[i] = reinterpret_cast<const int4*>(p.plan.rows(t) + r0)[i];
    };
    int t = 0, cg = 0;
    if (u0 < u1) {
      t = static_cast<int>(u0 % un.tiles);
      cg = static_cast<int>(u0 / un.tiles);
      look_ahead(t);
    }
    for (int64_t u = u0; good && u < u1; ++u) {
      const int side = cg >= un.cg0;
      const int64_t c0 = static_cast<int64_t>(cg - (side ? un.cg0 : 0)) * LORA_WG_COLS;
      const int C = static_cast<int>(side ? p.cols[1] : p.cols[0]);
      const uint16_t* X = side ? p.X[1] : p.X[0];
      const int rows_in = (ahead_n + LORA_WG_ROWS - 1) / LORA_WG_ROWS * LORA_WG_ROWS;   // rows past the count are zeros, up to the next MMA block
      int rows[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        rows[4 * i] = ahead[i].x; rows[4 * i + 1] = ahead[i].y; rows[4 * i + 2] = ahead[i].z; rows[4 * i + 3] = ahead[i].w;
      }
      if (++t == un.tiles) {
        t = 0;
        ++cg;
      }
      if (u + 1 < u1) look_ahead(t);
      for (int g = 0; g < 2 && c0 + g * 128 < C; ++g) {
        good = mbar_wait_warp(&empty_bar[stage], phase ^ 1u, abort_flag);
        if (!good) break;
        const uint32_t d = smem_u32(sX(stage)) + off;
        const int col = static_cast<int>(c0) + g * 128 + 8 * c;
        const int most = col < C ? static_cast<int>(p.plan.M) : 0;   // rows from here on are zeros
        const uint8_t* x = reinterpret_cast<const uint8_t*>(X + col);
        if (r0 < rows_in) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            cp_async16_or_zero(d + 128u * i + (((c & 7) ^ (i & 7)) << 4), x + row_bytes(rows[i], 2 * C), rows[i] < most);
        }
        cp_async_arrive(&full_bar[stage]);
        if (++stage == S::STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp == 4) {
    if (lane == 0) {
      // ---------------- MMA issuer ----------------
      const uint32_t idesc = idesc_f16(128, ALL ? static_cast<int>(G_COLS) : (p.R + 15) / 16 * 16, true) | IDESC_A_MN | IDESC_B_MN;
      int stage = 0, gb = 0, chain = 0;   // tiles in the accumulators
      uint32_t phase = 0, g_phase = 0, acc_phase = 0;   // a bit for each accumulator
      bool good = injected_wait(drain_bar, abort_flag);
      int t = 0, cg = 0;
      int2 info = make_int2(0, 0);
      if (u0 < u1) {
        t = static_cast<int>(u0 % un.tiles);
        cg = static_cast<int>(u0 / un.tiles);
        info = p.plan.info(t);
      }
      for (int64_t u = u0; good && u < u1; ++u) {
        const int side = cg >= un.cg0;
        const int64_t c0 = static_cast<int64_t>(cg - (side ? un.cg0 : 0)) * LORA_WG_COLS;
        const int2 here = info;
        const bool last = ++t == un.tiles;   // of these columns
        if (last) {
          t = 0;
          ++cg;
        }
        if (u + 1 < u1) info = p.plan.info(t);   // looked up a unit ahead
        const bool more_tiles = chain > 0;
        const bool close = ++chain == CHAIN || u + 1 == u1 || last || info.x != here.x;
        const int cols = c0 + 128 < (side ? p.cols[1] : p.cols[0]) ? 2 : 1;   // MMAs of 128 columns
#pragma unroll 1
        for (int b = 0; b < LORA_TILE / S::G_ROWS; ++b) {   // buffers of G
          if (S::G_ROWS * b >= here.y) break;
          good = mbar_wait(&gfull_bar[gb], g_phase, abort_flag);
          for (int g = 0; good && g < cols; ++g) {
            const int at = stage + g < S::STAGES ? stage + g : stage + g - S::STAGES;
            const uint32_t d = tmem_base + static_cast<uint32_t>(g) * G_COLS;
            if (b == 0) {
              if (!more_tiles) {
                good = mbar_wait(&tempty_bar[g], (acc_phase >> g & 1u) ^ 1u, abort_flag);
                acc_phase ^= 1u << g;
              }
              good = good && mbar_wait(&full_bar[at], stage + g < S::STAGES ? phase : phase ^ 1u, abort_flag);
              if (!good) break;
            }
            fence_proxy_async_smem();   // X and G were written by cp.async, through the generic proxy
            tc_fence_after();
            constexpr int KS = LORA_WG_ROWS / 16;
#pragma unroll
            for (int h = 0; h < S::G_ROWS / LORA_WG_ROWS; ++h) {
              const int row = S::G_ROWS * b + LORA_WG_ROWS * h;
              if (row >= here.y) break;
              const uint64_t adesc = sdesc_mn128(smem_u32(sX(at)) + row * 128, LORA_TILE * 128);
              const uint64_t bdesc = sdesc_mn128(smem_u32(sG(gb)) + h * (LORA_WG_ROWS * 128), ALL ? S::G_BYTES : S::G_ROWS * 128);
              const uint32_t more = more_tiles || row > 0 ? 1u : 0u;
#pragma unroll
              for (int k = 0; k < (ALL ? 1 : 3) * KS; ++k) {   // the parts of G: side by side, or the smallest first
                const int part = ALL ? 0 : 2 - k / KS;
                umma<2>(d, adesc + 128u * (k % KS), bdesc + 128u * (k % KS) + part * (S::G_BYTES >> 4), idesc, k == 0 ? more : 1u);
              }
            }
            if (S::G_ROWS * (b + 1) >= here.y) {   // the tile's last rows
              umma_commit(&empty_bar[at]);
              if (close) umma_commit(&tfull_bar[g]);
            }
          }
          if (!good) break;
          umma_commit(&gempty_bar[gb]);
          if (++gb == S::G_BUFS) { gb = 0; g_phase ^= 1u; }
        }
        stage += cols;
        if (stage >= S::STAGES) { stage -= S::STAGES; phase ^= 1u; }
        if (close) chain = 0;
      }
      drain_mma(drain_bar);
    }
  } else if (warp < 9) {
    // ---------------- zeros for adapters without rows; then the epilogue, once per segment ----------------
    const int L = static_cast<int>(p.plan.L);
    for (int a0 = 0; a0 < L; a0 += 32)
    for (uint32_t empty = __ballot_sync(0xffffffffu, a0 + lane < L && (un.tiles == 0 || p.plan.tile0()[a0 + lane] == p.plan.tile0()[a0 + lane + 1]));
         empty != 0; empty &= empty - 1) {
      const int a = a0 + __ffs(empty) - 1;
      for (int side = 0; side < 2; ++side) {
        // an adapter's dA or dB is contiguous: 16-byte pieces, dealt out over the CTAs
        const int64_t pieces = (side ? p.cols[1] : p.cols[0]) * p.R / 8;
        uint4* out = reinterpret_cast<uint4*>(side ? p.out[1] : p.out[0]) + a * pieces;
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x - 32 * 5; i < pieces; i += static_cast<int64_t>(gridDim.x) * 128)
          out[i] = make_uint4(0, 0, 0, 0);
      }
    }
    const int q = warp & 3;
    const uint32_t tmem = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    uint32_t acc_phase = 0;   // a bit for each accumulator
    bool good = true;
    for (int64_t u = u0; good && u < u1;) {   // one segment: the tiles of an adapter in this CTA's range, under one group of columns
      const int cg = static_cast<int>(u / un.tiles), t = static_cast<int>(u % un.tiles);
      const int side = cg >= un.cg0;
      const int64_t c0 = static_cast<int64_t>(cg - (side ? un.cg0 : 0)) * LORA_WG_COLS;
      const int a = p.plan.info(t).x;
      const int64_t seg0 = static_cast<int64_t>(cg) * un.tiles + p.plan.tile0()[a];
      const int64_t seg1 = static_cast<int64_t>(cg) * un.tiles + p.plan.tile0()[a + 1];
      const int64_t C = (side ? p.cols[1] : p.cols[0]), end = seg1 < u1 ? seg1 : u1;
      const bool whole = seg0 >= u0 && seg1 <= u1;
      const float s = side ? __ldg(p.scale + a) : 1.0f;
      float* part = p.part + (static_cast<int64_t>(blockIdx.x) * 2 + (seg0 >= u0 ? 1 : 0)) * p.R * LORA_WG_COLS;
      for (int64_t v0 = u; good && v0 < end; v0 += CHAIN) {
        const bool first = v0 == u, last = v0 + CHAIN >= end;
        for (int g = 0; g < 2 && c0 + g * 128 < C; ++g) {
          good = mbar_wait_warp(&tfull_bar[g], acc_phase >> g & 1u, abort_flag);
          if (!good) break;
          acc_phase ^= 1u << g;
          tc_fence_after();
          const int64_t col = c0 + g * 128 + q * 32 + lane;
          const uint32_t at = tmem + static_cast<uint32_t>(g) * G_COLS, sums = tmem + SUMS + static_cast<uint32_t>(g) * SUM_COLS;
          for (int c = 0; c < p.R; c += 16) {
            uint32_t v[16];
            __syncwarp();
            tmem_ld16(at + static_cast<uint32_t>(c), v);
            tmem_wait16(v);
            auto add = [&](uint32_t from) {
              uint32_t w[16];
              tmem_ld16(from + static_cast<uint32_t>(c), w);
              tmem_wait16(w);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
            };
            if constexpr (ALL) {
              add(at + 64);
              add(at + 128);
            }
            if (!first) add(sums);
            if (!last) {
              tmem_st16(sums + static_cast<uint32_t>(c), v);
              continue;
            }
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
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty_bar[g]);
        }
      }
      u = end;
    }
  } else {
    // ---------------- copies of G's parts, one tile a unit: chunk c of rows r0, r0 + step, ... of all parts ----------------
    constexpr int CH = RB * 8;                 // 16-byte chunks of a row of a part
    constexpr int STEP = 128 / CH, PER = LORA_TILE / STEP;
    const int ct = threadIdx.x - 32 * 9;
    const int c = ct % CH, r0 = ct / CH;
    const uint32_t off = static_cast<uint32_t>((c >> 3) * (S::G_ROWS * 128) + r0 * 128);
    int gb = 0, t = 0, cg = 0, n = 0;
    uint32_t g_phase = 0;
    int row[PER];   // the thread's rows of a unit, looked up a unit ahead; -1 past the count
    auto look_up = [&]() {
      n = p.plan.info(t).y;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        row[i] = p.plan.rows(t)[r0 + STEP * i];
        if (r0 + STEP * i >= n) row[i] = -1;
      }
    };
    if (u0 < u1) {
      t = static_cast<int>(u0 % un.tiles);
      cg = static_cast<int>(u0 / un.tiles);
      look_up();
    }
    for (int64_t u = u0; u < u1; ++u) {
      const uint16_t* G = cg >= un.cg0 ? p.G[1] : p.G[0];
      const int n64 = (n + LORA_WG_ROWS - 1) / LORA_WG_ROWS * LORA_WG_ROWS;
      bool good = true;
#pragma unroll
      for (int b = 0; b < LORA_TILE / S::G_ROWS; ++b) {
        if (S::G_ROWS * b >= n) break;
        good = mbar_wait_warp(&gempty_bar[gb], g_phase ^ 1u, abort_flag);
        if (!good) break;
        const uint32_t d = smem_u32(sG(gb)) + off;
#pragma unroll
        for (int i = 0; i < S::G_ROWS / STEP; ++i) {
          const int r = r0 + STEP * i, m = row[b * (S::G_ROWS / STEP) + i];   // row of the buffer, and of the batch
          if (S::G_ROWS * b + r < n64) {
            const bool on = m >= 0 && 8 * c < p.R;
            const uint16_t* src = G + row_bytes(m, 3 * p.R) + 8 * c;   // in elements
            const uint32_t at = d + 128u * STEP * i + (((c & 7) ^ (r & 7)) << 4);
#pragma unroll
            for (int j = 0; j < 3; ++j) cp_async16_or_zero(at + j * S::G_BYTES, src + j * p.R, on);
          }
        }
        cp_async_arrive(&gfull_bar[gb]);
        if (++gb == S::G_BUFS) { gb = 0; g_phase ^= 1u; }
      }
      if (!good) break;
      if (++t == un.tiles) {
        t = 0;
        ++cg;
      }
      if (u + 1 < u1) look_up();
    }
    cp_async_commit();
    cp_async_wait<0>();
  }
  __syncthreads();
  if (warp == 4) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, TCOLS);
  }
}

// The segments k_lora_wgrad cut between CTAs, added in CTA order. A CTA takes 8 values of R of 256 columns; blockIdx.x
// names the boundary between two CTAs' ranges.
__global__ void __launch_bounds__(LORA_WG_COLS) k_lora_wgrad_join(const LoraWgradParams p) {
  using T = __nv_bfloat16;
  griddep_wait();
  const LoraWgradUnits un(p);
  const int r0 = static_cast<int>(blockIdx.y) * 8, c1 = static_cast<int>(blockIdx.x);
  auto write = [&](int a, int cg, const float (&f)[8]) {
    const int side = cg >= un.cg0;
    const int64_t C = (side ? p.cols[1] : p.cols[0]), col = static_cast<int64_t>(cg - (side ? un.cg0 : 0)) * LORA_WG_COLS + threadIdx.x;
    if (col >= C) return;
    if (side == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p.out[0][(static_cast<int64_t>(a) * p.R + r0 + i) * C + col] = from_f<T>(f[i]);
    } else {
      *reinterpret_cast<uint4*>(p.out[1] + (static_cast<int64_t>(a) * C + col) * p.R + r0) = narrow8<T>(f);
    }
  };
  // the segment that CTA c1 - 1 leaves to CTA c1, if it began in c1 - 1
  if (c1 > 0 && c1 < un.ctas) {
    const int64_t u = un.first(c1);
    const int cg = static_cast<int>(u / un.tiles), t = static_cast<int>(u % un.tiles), a = p.plan.info(t).x;
    const int64_t s0 = u - t + p.plan.tile0()[a], s1 = u - t + p.plan.tile0()[a + 1];
    if (s0 < u && un.first(c1 - 1) <= s0) {
      float f[8] = {};
      for (int c = c1 - 1; c < un.ctas && un.first(c) < s1; ++c) {
        const float* part = p.part + (static_cast<int64_t>(c) * 2 + (un.first(c) <= s0 ? 1 : 0)) * p.R * LORA_WG_COLS;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += part[(r0 + i) * LORA_WG_COLS + threadIdx.x];
      }
      const float s = cg >= un.cg0 ? __ldg(p.scale + a) : 1.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= s;
      write(a, cg, f);
    }
  }
}

}  // namespace qlin
