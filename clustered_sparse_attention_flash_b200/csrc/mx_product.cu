// Product of two microscaled 4-bit matrices on the tensor cores:
//   Y[m][n] = sum_k A[m][k] W[n][k] + bias[n]
// A [M][K] tokens, W [N][K] features, both MXFP4 (mx_quant.cu), Y bf16.
//
// tcgen05.mma kind::mxf4 multiplies E2M1 pairs exactly and applies one E8M0
// scale per 32 elements of each operand; sums are float32 in tensor memory and
// rounded once, to bf16.  The features are the MMA's 128 rows and the tokens
// its columns, so that the tile narrows to 16 columns for a few tokens while
// the weights still stream through full tiles.
//
// One persistent block per SM:
//   warp 0       TMA: code tiles of 256 elements (128 bytes per row, 128-byte
//                swizzle) into a ring of stages
//   warp 1       tensor memory, copies of the scales into it, MMAs
//   warps 4-7    scales: plain rows in global memory to the tensor core's
//                order in shared memory (a 128-row, 4-scale atom is 512 bytes,
//                row r at 16 (r mod 32) + 4 (r div 32))
//   warps 8-11   epilogue: accumulators + bias to bf16 through shared memory
//                into coalesced rows; two accumulators, so that it runs
//                beside the next tile's MMAs
// Scales keep one tensor-memory slot per ring stage: a slot is written again
// only after the MMAs that read it have committed.
#include <cuda.h>

#include <algorithm>

#include "internal.h"
#include "tc_common.cuh"

namespace svg {

namespace {

constexpr int kThreads = 384;
constexpr int kTF = 128;          // features per tile (MMA M)
constexpr int kKB = 256;          // elements of K per stage (128 bytes of codes)
constexpr int kChunk = 32;        // tokens per epilogue step
constexpr int kSmemLimit = 232448;

// Tile of TN tokens (MMA N).
template <int TN>
struct Tile {
  static constexpr int kTokBlocks = (TN + 127) / 128;        // 128-row scale atoms of the tokens
  static constexpr int kCodesF = kTF * 128, kCodesT = TN * 128;
  static constexpr int kSfF = 2 * 512, kSfT = 2 * 512 * kTokBlocks;
  static constexpr int kStage = kCodesF + kCodesT + kSfF + kSfT;
  static constexpr int kStages = TN > 128 ? 4 : TN > 64 ? 5 : 6;
  static constexpr int kOut = 2 * kChunk * kTF * 2;          // two staging buffers, bf16
  static constexpr int kBars = 256;
  static constexpr int kSmem = kStages * kStage + kOut + kBars + 1024;
  static constexpr int kAccCols = TN;                        // per accumulator, two of them
  static constexpr int kSfCols = 8 + 8 * kTokBlocks;         // per stage: 2 atoms of features, 2 of each token block
  static constexpr int kCols = 2 * kAccCols + kStages * kSfCols;
  static constexpr int kAlloc = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512 && kSmem <= kSmemLimit, "tile does not fit");
};

struct ProductArgs {
  const uint8_t *a_scales, *w_scales;
  const float* bias;
  bf16* Y;
  int M, N, K, ftiles, tiles, kblocks;
  int* status;
};

// kind::mxf4, both operands E2M1, scales E8M0 (one per 32), M x N tile; ids
// select the first or second scale pair of a 4-byte column.
__host__ __device__ constexpr uint32_t idesc_mxf4(int N, uint32_t id) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | (1u << 27) | (id << 4) | (id << 29);
}

__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// One scale atom (32 rows of 16 bytes in shared memory) into 4 tensor-memory
// columns, for all four lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(tc::sdesc(saddr, 128, 128, 0))
               : "memory");
}

// Scales [16 u, 16 u + 16) of a row with `pitch` scales (two stages); 0 behind
// the end.  As wide as the rows are aligned.
__device__ __forceinline__ uint4 load_scales(const uint8_t* row, int pitch, int u) {
  const uint8_t* s = row + u * 16;
  if ((pitch & 15) == 0) return __ldg(reinterpret_cast<const uint4*>(s));
  uint32_t v[4] = {0, 0, 0, 0};
  const int left = pitch - u * 16;
  if ((pitch & 3) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * i < left) v[i] = __ldg(reinterpret_cast<const uint32_t*>(s) + i);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < left) v[i >> 2] |= (uint32_t)__ldg(s + i) << (8 * (i & 3));
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

template <int TN>
__global__ void __launch_bounds__(kThreads, 1)
    k_mx_product(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a, const ProductArgs p) {
  using T = Tile<TN>;
  constexpr int S = T::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // code tiles first (1,024-byte aligned), then the scales of all stages, then the output staging
  uint8_t* codes_s = smem;
  uint8_t* sf_s = smem + S * (T::kCodesF + T::kCodesT);
  bf16* out_s = reinterpret_cast<bf16*>(sf_s + S * (T::kSfF + T::kSfT));
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(out_s) + T::kOut);
  uint64_t* codes_full = bars;            // [S]
  uint64_t* sf_full = bars + S;           // [S]
  uint64_t* empty = bars + 2 * S;         // [S]
  uint64_t* acc_full = bars + 3 * S;      // [2]
  uint64_t* acc_empty = bars + 3 * S + 2; // [2]
  uint64_t* done = bars + 3 * S + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * S + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 3 * S + 6);
  volatile int* no_flag = abort_flag + 1;  // stays 0: waits that an abort must not cut short
  static_assert((3 * S + 7) * 8 <= T::kBars, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      tc::mbar_init(codes_full + i, 1);
      tc::mbar_init(sf_full + i, 4);
      tc::mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(acc_full + i, 1);
      tc::mbar_init(acc_empty + i, 4);
    }
    tc::mbar_init(done, 1);
    *abort_flag = 0;
    *no_flag = 0;
    tc::mbar_fence_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, T::kAlloc);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------- code tiles
    if (lane == 0) {
      tc::tma_prefetch_map(&map_w);
      tc::tma_prefetch_map(&map_a);
      uint32_t it = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < p.tiles; t += gridDim.x) {
        const int f0 = t % p.ftiles * kTF, m0 = t / p.ftiles * TN;
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const int s = it % S;
          ok = tc::mbar_wait(empty + s, (it / S & 1) ^ 1, abort_flag, p.status);
          if (!ok) break;
          const uint32_t dst = tc::smem_u32(codes_s + s * (T::kCodesF + T::kCodesT));
          tc::mbar_arrive_expect_tx(codes_full + s, T::kCodesF + T::kCodesT);
          tc::tma_load_3d(dst, &map_w, kb * (kKB / 2), f0, 0, codes_full + s);
          tc::tma_load_3d(dst + T::kCodesF, &map_a, kb * (kKB / 2), m0, 0, codes_full + s);
        }
      }
      // The block's memory outlives its copies, also after an abort.
      for (uint32_t i = it > S ? it - S : 0; i < it; ++i) tc::mbar_wait(codes_full + i % S, i / S & 1, no_flag, p.status);
    }
    __syncwarp();
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMAs
    const bool leader = tc::elect_one();
    uint32_t it = 0, n = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < p.tiles; t += gridDim.x, ++n) {
      const uint32_t buf = n & 1, acc = tmem + buf * T::kAccCols;
      ok = tc::mbar_wait_warp(acc_empty + buf, (n >> 1 & 1) ^ 1, abort_flag, p.status);
      for (int kb = 0; ok && kb < p.kblocks; ++kb, ++it) {
        const int s = it % S;
        ok = tc::mbar_wait_warp(codes_full + s, it / S & 1, abort_flag, p.status) &&
             tc::mbar_wait_warp(sf_full + s, it / S & 1, abort_flag, p.status);
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t wf = tc::smem_u32(codes_s + s * (T::kCodesF + T::kCodesT)), tk = wf + T::kCodesF;
        const uint32_t sf = tc::smem_u32(sf_s + s * (T::kSfF + T::kSfT));
        const uint32_t tf = tmem + 2 * T::kAccCols + s * T::kSfCols, tt = tf + 8;
        if (leader) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            copy_scales(tf + i * 4, sf + i * 512);
#pragma unroll
            for (int b = 0; b < T::kTokBlocks; ++b)
              copy_scales(tt + (i * T::kTokBlocks + b) * 4, sf + T::kSfF + (i * T::kTokBlocks + b) * 512);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_mxf4(acc, tc::desc_kmajor(wf, 0, k), tc::desc_kmajor(tk, 0, k), idesc_mxf4(TN, (k & 1) * 2), tf + (k >> 1) * 4,
                     tt + (k >> 1) * T::kTokBlocks * 4, (kb | k) ? 1u : 0u);
          tc::mma_commit(empty + s);
          if (kb + 1 == p.kblocks) tc::mma_commit(acc_full + buf);
        }
        __syncwarp();
      }
    }
    if (leader) tc::mma_commit(done);
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ scales
    // Row r of the features and rows r, r + 128 of the tokens.  A load takes the
    // scales of two stages and runs two loads (two to four stages) ahead of
    // the stores, over tile boundaries too.
    const int r = threadIdx.x - 128;
    const int pitch = p.K / 32, units = (p.kblocks + 1) / 2;
    constexpr int R = T::kTokBlocks;
    struct Unit {
      uint4 v[R + 1];
    };
    int ft = blockIdx.x, fu = 0;  // the next unit to load
    auto fetch = [&](Unit& x) {
      const int f = ft % p.ftiles * kTF + r, m0 = ft / p.ftiles * TN;
      const bool more = ft < p.tiles;
      x.v[0] = more && f < p.N ? load_scales(p.w_scales + (size_t)f * pitch, pitch, fu) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int b = 0; b < R; ++b) {
        const int m = r + b * 128;
        x.v[b + 1] = more && m < TN && m0 + m < p.M ? load_scales(p.a_scales + (size_t)(m0 + m) * pitch, pitch, fu) : make_uint4(0, 0, 0, 0);
      }
      if (++fu == units) {
        fu = 0;
        ft += gridDim.x;
      }
    };
    uint32_t it = 0;
    bool ok = true;
    auto store = [&](const Unit& x, int h) {
      const int s = it % S;
      ok = tc::mbar_wait_warp(empty + s, (it / S & 1) ^ 1, abort_flag, p.status);
      if (!ok) return;
      uint8_t* sf = sf_s + s * (T::kSfF + T::kSfT) + (r & 31) * 16 + (r >> 5) * 4;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<uint32_t*>(sf + i * 512) = h ? (i ? x.v[0].w : x.v[0].z) : (i ? x.v[0].y : x.v[0].x);
#pragma unroll
        for (int b = 0; b < R; ++b)
          *reinterpret_cast<uint32_t*>(sf + T::kSfF + (i * R + b) * 512) =
              h ? (i ? x.v[b + 1].w : x.v[b + 1].z) : (i ? x.v[b + 1].y : x.v[b + 1].x);
      }
      tc::fence_proxy_async();  // the tensor core's copies read what this thread stored
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(sf_full + s);
      ++it;
    };
    Unit x0, x1, x2;
    fetch(x0);
    fetch(x1);
    for (int t = blockIdx.x; ok && t < p.tiles; t += gridDim.x)
      for (int u = 0; ok && u < units; ++u) {
        fetch(x2);
        store(x0, 0);
        if (ok && 2 * u + 1 < p.kblocks) store(x0, 1);
        x0 = x1;
        x1 = x2;
      }
  } else if (warp >= 8) {
    // ---------------------------------------------------------- epilogue
    const int quarter = warp & 3, f = quarter * 32 + lane, tid = threadIdx.x - 256;
    constexpr int C = TN < kChunk ? TN : kChunk;
    uint32_t n = 0, step = 0;
    for (int t = blockIdx.x; t < p.tiles; t += gridDim.x, ++n) {
      const int f0 = t % p.ftiles * kTF, m0 = t / p.ftiles * TN;
      const uint32_t buf = n & 1;
      const float bias = p.bias && f0 + f < p.N ? p.bias[f0 + f] : 0.f;
      if (!tc::bar_and(1, 128, tc::mbar_wait_warp(acc_full + buf, n >> 1 & 1, abort_flag, p.status))) break;
      tc::tc_fence_after();
      const int rows = min(TN, p.M - m0);
      for (int c = 0; c < TN; c += C, ++step) {
        if (c >= rows) break;  // uniform: tokens behind the last one
        uint32_t v[32];
        const uint32_t at = tc::taddr(tmem, quarter * 32, buf * T::kAccCols + c);
        if constexpr (C == 32) {
          tc::tmem_ld32(at, v);
        } else {
          uint32_t w[16];
          tc::tmem_ld16(at, w);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = w[i];
        }
        tc::tmem_ld_wait();
        bf16* st = out_s + (step & 1) * (kChunk * kTF);
#pragma unroll
        for (int i = 0; i < C; ++i) st[i * kTF + f] = __float2bfloat16_rn(__uint_as_float(v[i]) + bias);
        asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
        for (int u = 0; u < C / 8; ++u) {
          const int e = u * 128 + tid, m = e >> 4, col = (e & 15) * 8;
          if (c + m < rows && f0 + col < p.N)
            *reinterpret_cast<uint4*>(p.Y + (size_t)(m0 + c + m) * p.N + f0 + col) = *reinterpret_cast<const uint4*>(st + m * kTF + col);
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(acc_empty + buf);
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::mbar_wait(done, 0, no_flag, p.status);
    __syncwarp();
    tc::tmem_dealloc(tmem, T::kAlloc);
  }
}

// ------------------------------------------------------------- few tokens
//
// Up to 64 tokens the product is a stream of the weights.  A cluster of C blocks
// shares a tile of 128 features: block r takes the r-th part of K, and the
// partial sums meet through distributed shared memory, added in rank order (no
// workspace, no atomics, the same bits every time).  C grows while the blocks
// stay at about one per SM and each has two stages: a second wave costs more
// than the split gains (us, one token, K = 5,120, C = 1 / 2 / 4 / 8: N = 5,120
// 11.3 / 8.7 / 8.7 / 12.2; N = 15,360 12.2 / 12.6 / 16.6 / 25.5).

constexpr int kFewThreads = 256;  // warp 0 TMA, 1 MMA, 4-7 scales, then the sums

template <int TN>
struct FewTile {
  static constexpr int kCodesF = kTF * 128, kCodesT = TN * 128;
  static constexpr int kCodes = kCodesF + kCodesT, kSf = 2048;  // 2 atoms each of features and tokens
  static constexpr int kStages = TN > 16 ? 4 : 5;
  static constexpr int kBars = 256;
  static constexpr int kSmem = kStages * (kCodes + kSf) + kBars + 1024;
  static constexpr int kSfCols = 16;
  static constexpr int kAlloc = TN + kStages * kSfCols <= 128 ? 128 : 256;
  static_assert(kStages * kCodes >= TN * kTF * 4, "partial sums take the ring's place");
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of every block of the cluster (warps converged).
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_address(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 load_peer(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Scales [8 kb, 8 kb + 8) of a row with `pitch` scales (one stage); 0 behind the end.
__device__ __forceinline__ uint2 load_scales8(const uint8_t* row, int pitch, int kb) {
  const uint8_t* s = row + kb * 8;
  if ((pitch & 7) == 0) return __ldg(reinterpret_cast<const uint2*>(s));
  const int left = pitch - kb * 8;
  uint32_t v[2] = {0, 0};
  if ((pitch & 3) == 0) {
    v[0] = __ldg(reinterpret_cast<const uint32_t*>(s));
    if (left > 4) v[1] = __ldg(reinterpret_cast<const uint32_t*>(s) + 1);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) v[i >> 2] |= (uint32_t)__ldg(s + i) << (8 * (i & 3));
  }
  return make_uint2(v[0], v[1]);
}

template <int TN>
__global__ void __launch_bounds__(kFewThreads, 2)
    k_mx_few(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a, const ProductArgs p, int C) {
  using T = FewTile<TN>;
  constexpr int S = T::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* codes_s = smem;
  uint8_t* sf_s = smem + S * T::kCodes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sf_s + S * T::kSf);
  uint64_t* codes_full = bars;     // [S]
  uint64_t* sf_full = bars + S;    // [S]
  uint64_t* empty = bars + 2 * S;  // [S]
  uint64_t* done = bars + 3 * S;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * S + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 3 * S + 2);
  volatile int* no_flag = abort_flag + 1;  // stays 0: waits that an abort must not cut short
  static_assert((3 * S + 3) * 8 <= T::kBars, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = C > 1 ? (int)cluster_rank() : 0, tile = blockIdx.x / C;
  const int f0 = tile % p.ftiles * kTF, m0 = tile / p.ftiles * TN;
  const int kb0 = (int)((long long)rank * p.kblocks / C), kb1 = (int)((long long)(rank + 1) * p.kblocks / C);
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      tc::mbar_init(codes_full + i, 1);
      tc::mbar_init(sf_full + i, 4);
      tc::mbar_init(empty + i, 1);
    }
    tc::mbar_init(done, 1);
    *abort_flag = 0;
    *no_flag = 0;
    tc::mbar_fence_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, T::kAlloc);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------- code tiles
    if (lane == 0) {
      int it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % S;
        if (!tc::mbar_wait(empty + s, (it / S & 1) ^ 1, abort_flag, p.status)) break;
        const uint32_t dst = tc::smem_u32(codes_s + s * T::kCodes);
        tc::mbar_arrive_expect_tx(codes_full + s, T::kCodes);
        tc::tma_load_3d(dst, &map_w, kb * (kKB / 2), f0, 0, codes_full + s);
        tc::tma_load_3d(dst + T::kCodesF, &map_a, kb * (kKB / 2), m0, 0, codes_full + s);
      }
      // The block's memory outlives its copies, also after an abort.
      for (int i = max(it - S, 0); i < it; ++i) tc::mbar_wait(codes_full + i % S, i / S & 1, no_flag, p.status);
    }
    __syncwarp();
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMAs
    const bool leader = tc::elect_one();
    int it = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++it) {
      const int s = it % S;
      if (!(tc::mbar_wait_warp(codes_full + s, it / S & 1, abort_flag, p.status) &&
            tc::mbar_wait_warp(sf_full + s, it / S & 1, abort_flag, p.status)))
        break;
      tc::tc_fence_after();
      const uint32_t wf = tc::smem_u32(codes_s + s * T::kCodes), tk = wf + T::kCodesF;
      const uint32_t sf = tc::smem_u32(sf_s + s * T::kSf);
      const uint32_t tf = tmem + TN + s * T::kSfCols;
      if (leader) {
#pragma unroll
        for (int i = 0; i < 4; ++i) copy_scales(tf + i * 4, sf + i * 512);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_mxf4(tmem, tc::desc_kmajor(wf, 0, k), tc::desc_kmajor(tk, 0, k), idesc_mxf4(TN, (k & 1) * 2), tf + (k >> 1) * 4,
                   tf + 8 + (k >> 1) * 4, (it | k) ? 1u : 0u);
        tc::mma_commit(empty + s);
      }
      __syncwarp();
    }
    if (leader) tc::mma_commit(done);
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ scales
    // Row r of the features and of the tokens, four stages loaded ahead.
    const int r = threadIdx.x - 128, pitch = p.K / 32;
    const uint8_t* wrow = f0 + r < p.N ? p.w_scales + (size_t)(f0 + r) * pitch : nullptr;
    const uint8_t* arow = r < TN && m0 + r < p.M ? p.a_scales + (size_t)(m0 + r) * pitch : nullptr;
    constexpr int B = 4;
    uint2 cw[B], ca[B], nw[B], na[B];
    auto fetch = [&](int kb, uint2 (&w)[B], uint2 (&a)[B]) {
#pragma unroll
      for (int i = 0; i < B; ++i) {
        w[i] = wrow && kb + i < kb1 ? load_scales8(wrow, pitch, kb + i) : make_uint2(0, 0);
        a[i] = arow && kb + i < kb1 ? load_scales8(arow, pitch, kb + i) : make_uint2(0, 0);
      }
    };
    fetch(kb0, cw, ca);
    bool ok = true;
    for (int kb = kb0; ok && kb < kb1; kb += B) {
      fetch(kb + B, nw, na);
#pragma unroll
      for (int i = 0; i < B; ++i) {
        if (!ok || kb + i >= kb1) break;
        const int it = kb + i - kb0, s = it % S;
        ok = tc::mbar_wait_warp(empty + s, (it / S & 1) ^ 1, abort_flag, p.status);
        if (!ok) break;
        uint8_t* sf = sf_s + s * T::kSf + (r & 31) * 16 + (r >> 5) * 4;
        *reinterpret_cast<uint32_t*>(sf) = cw[i].x;
        *reinterpret_cast<uint32_t*>(sf + 512) = cw[i].y;
        *reinterpret_cast<uint32_t*>(sf + 1024) = ca[i].x;
        *reinterpret_cast<uint32_t*>(sf + 1536) = ca[i].y;
        tc::fence_proxy_async();  // the tensor core's copies read what this thread stored
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(sf_full + s);
      }
#pragma unroll
      for (int i = 0; i < B; ++i) {
        cw[i] = nw[i];
        ca[i] = na[i];
      }
    }
    // -------------------------------------------------------------- sums
    const int quarter = warp & 3, f = quarter * 32 + lane, rows = min(TN, p.M - m0);
    const float bias = p.bias && f0 + f < p.N ? p.bias[f0 + f] : 0.f;
    ok = tc::mbar_wait_warp(done, 0, abort_flag, p.status) && ok;
    tc::tc_fence_after();
    float* part = reinterpret_cast<float*>(codes_s);  // [TN][128], in the ring's place: every MMA has read it
    if (ok)
#pragma unroll
      for (int c = 0; c < TN; c += 16) {
        uint32_t v[16];
        tc::tmem_ld16(tc::taddr(tmem, quarter * 32, c), v);
        tc::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (C > 1) part[(c + i) * kTF + f] = __uint_as_float(v[i]);
          else if (c + i < rows && f0 + f < p.N) p.Y[(size_t)(m0 + c + i) * p.N + f0 + f] = __float2bfloat16_rn(__uint_as_float(v[i]) + bias);
        }
      }
    if (C > 1) {
      __syncwarp();
      cluster_sync();
      // This block sums the tokens rank, rank + C, ...: four features a thread,
      // the loads of four (token, features) from one peer in flight together.
      const uint32_t at = tc::smem_u32(part);
      const int mine = rows > rank ? (rows - rank + C - 1) / C : 0, col = lane * 4;
      for (int j0 = quarter; ok && j0 < mine && f0 + col < p.N; j0 += 16) {
        float4 s[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) s[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < C; ++i) {
          const uint32_t peer = peer_address(at, i);
          float4 v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) v[u] = load_peer(peer + ((rank + min(j0 + 4 * u, mine - 1) * C) * kTF + col) * 4);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            s[u].x += v[u].x; s[u].y += v[u].y; s[u].z += v[u].z; s[u].w += v[u].w;
          }
        }
        const float4 b = p.bias ? *reinterpret_cast<const float4*>(p.bias + f0 + col) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (j0 + 4 * u < mine) {
            __nv_bfloat162 y[2] = {__floats2bfloat162_rn(s[u].x + b.x, s[u].y + b.y), __floats2bfloat162_rn(s[u].z + b.z, s[u].w + b.w)};
            *reinterpret_cast<uint2*>(p.Y + (size_t)(m0 + rank + (j0 + 4 * u) * C) * p.N + f0 + col) = *reinterpret_cast<const uint2*>(y);
          }
      }
      __syncwarp();
    }
  }
  if (C > 1) {
    if (warp < 4) {
      __syncwarp();
      cluster_sync();
    }
    cluster_sync();  // a block's partial sums stay until every block has read them
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::mbar_wait(done, 0, no_flag, p.status);
    __syncwarp();
    tc::tmem_dealloc(tmem, T::kAlloc);
  }
}

template <int TN>
cudaError_t launch_few(ProductArgs p, const uint8_t* a_codes, const uint8_t* w_codes, cudaStream_t st) {
  using T = FewTile<TN>;
  CUtensorMap map_w, map_a;
  if (!tma_map_u8_rows(&map_w, w_codes, p.K / 2, p.N, kTF) || !tma_map_u8_rows(&map_a, a_codes, p.K / 2, p.M, TN))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(k_mx_few<TN>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
  if (e != cudaSuccess) return e;
  p.ftiles = (p.N + kTF - 1) / kTF;
  p.tiles = p.ftiles * ((p.M + TN - 1) / TN);
  int C = 1;
  while (C < 8 && p.tiles * C * 2 <= 160 && p.kblocks >= 4 * C) C *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.tiles * C);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = T::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k_mx_few<TN>, map_w, map_a, p, C);
  note_launch();
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int TN>
cudaError_t launch(ProductArgs p, const uint8_t* a_codes, const uint8_t* w_codes, cudaStream_t st) {
  using T = Tile<TN>;
  CUtensorMap map_w, map_a;
  if (!tma_map_u8_rows(&map_w, w_codes, p.K / 2, p.N, kTF) || !tma_map_u8_rows(&map_a, a_codes, p.K / 2, p.M, TN))
    return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(k_mx_product<TN>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
  if (e != cudaSuccess) return e;
  p.ftiles = (p.N + kTF - 1) / kTF;
  p.tiles = p.ftiles * ((p.M + TN - 1) / TN);
  k_mx_product<TN><<<std::min(p.tiles, 148), kThreads, T::kSmem, st>>>(map_w, map_a, p);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

size_t mx_product_ws_bytes(int M, int N, int K) {
  (void)M; (void)N; (void)K;
  return 0;
}

cudaError_t mx_product_run(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* w_codes, const uint8_t* w_scales,
                           const float* bias, int M, int N, int K, void* Y, void* ws, cudaStream_t st) {
  (void)ws;
  ProductArgs p{};
  p.a_scales = a_scales; p.w_scales = w_scales; p.bias = bias;
  p.Y = static_cast<bf16*>(Y);
  p.M = M; p.N = N; p.K = K;
  p.kblocks = (K + kKB - 1) / kKB;
  p.status = status_word();
  if (!p.status) return cudaErrorInvalidValue;
  if (M <= 16) return launch_few<16>(p, a_codes, w_codes, st);
  // From 65 tokens on the wide tiles win even where they leave SMs idle (256 tokens, N = K = 5,120: 15.0 us
  // against 17.4 us in tiles of 64).
  if (M <= 64) return launch_few<64>(p, a_codes, w_codes, st);
  return launch<192>(p, a_codes, w_codes, st);
}

}  // namespace svg
