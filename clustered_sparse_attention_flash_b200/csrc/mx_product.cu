// Product of two microscaled 4-bit matrices on the tensor cores:
//   Y[m][n] = sum_k A[m][k] W[n][k] + bias[n]
// A [M][K] tokens, W [N][K] features, both MXFP4 (mx_quant.cu), Y bf16.
//
// tcgen05.mma kind::mxf4 multiplies E2M1 pairs exactly and applies one E8M0
// scale per 32 elements of each operand; sums are float32 in tensor memory and
// rounded once, to bf16.  The features are the MMA's rows and the tokens its
// columns, so that the tile narrows to 16 columns for a few tokens while the
// weights still stream through full tiles.
//
// Scales lie as plain rows in global memory.  A warpgroup brings them into the
// tensor core's order in shared memory (an atom of 128 rows x 4 scales is 512
// bytes, row r at 16 (r mod 32) + 4 (r div 32)), from where tcgen05.cp takes
// them to tensor memory, into a slot that is written again only after the MMAs
// that read it have committed.
#include <cuda.h>

#include <algorithm>

#include "chain.cuh"
#include "internal.h"
#include "tc_common.cuh"

namespace svg {

namespace {

constexpr int kTF = 128;          // features per block
constexpr int kKB = 256;          // elements of K per stage (128 bytes of codes)
constexpr int kChunk = 32;        // tokens per epilogue step
constexpr int kSmemLimit = 232448;

struct ProductArgs {
  const uint8_t *a_scales, *w_scales;
  const float* bias;
  bf16* Y;
  int M, N, K, ftiles, tiles, kblocks;
  int* status;
};

// kind::mxf4, both operands E2M1, scales E8M0 (one per 32), M x N tile; ids
// select the first or second scale pair of a 4-byte column.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, uint32_t id) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27) | (id << 4) | (id << 29);
}

__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// The row whose scales thread t of the scale warps stores: word t of an atom, so
// that a warp's stores meet no bank twice (row t itself would four times).
__device__ __forceinline__ int scale_row(int t) { return (t & 3) * 32 + (t >> 2); }

// One scale atom (32 rows of 16 bytes in shared memory) into 4 tensor-memory
// columns, for all four lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(tc::sdesc(saddr, 128, 128, 0))
               : "memory");
}

// Scales [16 u, 16 u + 16) of a row with `pitch` scales (two stages); 0 behind
// the end.  As wide as the rows are aligned, and coherent loads: the kernel ahead
// may write the scales while this one is already running (chain.cuh).
__device__ __forceinline__ uint4 load_scales(const uint8_t* row, int pitch, int u) {
  const uint8_t* s = row + u * 16;
  if ((pitch & 15) == 0) return *reinterpret_cast<const uint4*>(s);
  uint32_t v[4] = {0, 0, 0, 0};
  const int left = pitch - u * 16;
  if ((pitch & 3) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * i < left) v[i] = reinterpret_cast<const uint32_t*>(s)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < left) v[i >> 2] |= (uint32_t)s[i] << (8 * (i & 3));
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// ------------------------------------------------------------- many tokens
//
// Two neighbouring SMs work on one tile of 256 features x TN tokens
// (cta_group::2): each holds its own 128 features and half of the tokens, so
// that at TN = 192 an SM reads 7 KB of codes per 64 elements of K where a tile of
// its own would read 10 KB.  What bounds it is how fast an SM takes in codes, 66
// to 68 bytes per ns at every width (a stage of 256 elements of K is 20, 24, 28
// and 30 KB at TN = 64, 128, 192 and 224 and takes 300, 375, 435 and 461 ns), so
// a wider tile gains by its fewer bytes per product; and, at the largest sizes,
// the power limit.  No one unit is at its peak: tensor pipe 63 % busy, 48 bytes a
// clock from the L2 at 1.61 GHz.  75,600 x 15,360 x 5,120 of quantised normal data
// takes 2.53 ms at TN = 224 when the chip is cool, 4.7 PFLOP/s, 0.73 of four times
// the measured bf16 burst rate, and 2.8 ms in a row (0.65); with zeros for data,
// which take less power, 5.6 PFLOP/s.  (TN = 192: 2.72 ms; one SM per tile of
// 128 x 192: 3.47 ms.)  Beside two accumulators of 224 tokens tensor
// memory holds the scales of two stages, so that a stage's scales wait for the
// MMAs two stages back; narrower tiles have a slot for each stage of the ring.
// The launcher chooses by the rounds of tiles.  The even block issues the MMAs
// for both.
//   warp 0       TMA: code tiles of 256 elements (128 bytes per row, 128-byte
//                swizzle) into a ring of stages; both blocks' copies complete on
//                the even block's barrier
//   warp 1       tensor memory; in the even block scale copies and MMAs
//   warps 4-7    scales of the block's features and of all the tile's tokens, in
//                units of two stages and a ring of their own, eight units deep
//   warps 1-3    in the odd block: pass the word that an accumulator has been
//                read (1) or a unit is there (2, 3) on to the even block.  The
//                release over the cluster that this takes costs about a thousand
//                cycles (and would wait for the scale warps' loads in flight):
//                hence warps of their own and the deep ring.  (75,600 x 15,360 x
//                5,120: 6.61 ms with the scale warps releasing, 4.15 ms with a
//                ring of five stages, 2.82 ms so.)
//   warps 8-11   epilogue: accumulators + bias to bf16 through shared memory
//                into coalesced rows; two accumulators, so that it runs beside
//                the next tile's MMAs

constexpr int kPairThreads = 384;

template <int TN>
struct Pair {
  static constexpr int kTokBlocks = TN > 128 ? 2 : 1;              // 128-row scale atoms of the tokens
  static constexpr int kCodesF = kTF * 128, kCodesT = TN / 2 * 128, kCodes = kCodesF + kCodesT;
  static constexpr int kSfF = 2 * 512, kSf = kSfF + 2 * 512 * kTokBlocks;  // scales of a stage
  static constexpr int kStages = TN > 128 ? 5 : 7, kUnits = 8;
  static constexpr int kOut = 2 * kChunk * kTF * 2;                // two staging buffers, bf16
  static constexpr int kBars = 512;
  static constexpr int kSmem = kStages * kCodes + kUnits * 2 * kSf + kOut + kBars + 1024;
  static constexpr int kSfCols = 8 + 8 * kTokBlocks;               // per stage: 2 atoms of features, 2 of each token block
  static constexpr int kSfSlots = TN <= 192 ? kStages : 2;         // of tensor memory
  static_assert(2 * TN + kSfSlots * kSfCols <= 512 && kSmem <= kSmemLimit && kCodes % 1024 == 0, "tile does not fit");
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

// The address of a barrier of the even block.
__device__ __forceinline__ uint32_t leader_address(const uint64_t* bar) { return peer_address(tc::smem_u32(bar), 0); }
__device__ __forceinline__ void arrive_leader(const uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(leader_address(bar)) : "memory");
}
// tc::mbar_wait_warp for barriers that the other block arrives at.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  bool ok = false;
  const uint64_t t0 = tc::globaltimer();
  for (uint32_t it = 1;; ++it) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    if (done) {
      ok = true;
      break;
    }
    if ((it & 255u) == 0) {
      if (*abort_flag) break;
      if (tc::globaltimer() - t0 > tc::kWaitLimitNs) {
        set_status(status, ST_TIMEOUT);
        *abort_flag = 1;
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const void* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(0), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void copy_scales_pair(uint32_t taddr, uint32_t saddr) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(tc::sdesc(saddr, 128, 128, 0)) : "memory");
}
__device__ __forceinline__ void mma_mxf4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// Arrive on `bar` of both blocks once every MMA and copy issued so far is done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          tc::smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

template <int TN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    k_mx_pair(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a, const ProductArgs args) {
  using T = Pair<TN>;
  constexpr int S = T::kStages, U = T::kUnits;
  ProductArgs p = args;
  extern __shared__ uint8_t smem_raw[];
  // the dynamic part starts at the same offset in both blocks, and so does all of this
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* codes_s = smem;
  uint8_t* sf_s = smem + S * T::kCodes;
  bf16* out_s = reinterpret_cast<bf16*>(sf_s + U * 2 * T::kSf);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(out_s) + T::kOut);
  uint64_t* codes_full = bars;            // [S] of the even block: both blocks' codes
  uint64_t* empty = codes_full + S;       // [S]
  uint64_t* sf_full = empty + S;          // [U] own scales; in the even block the other's word too
  uint64_t* sf_empty = sf_full + U;       // [U]
  uint64_t* acc_full = sf_empty + U;      // [2]
  uint64_t* acc_empty = acc_full + 2;     // [2] own epilogue; in the even block the other's word too
  uint64_t* done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(done + 2);
  volatile int* no_flag = abort_flag + 1;  // stays 0: waits that an abort must not cut short
  static_assert((2 * S + 2 * U + 7) * 8 <= T::kBars, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      tc::mbar_init(codes_full + i, 1);
      tc::mbar_init(empty + i, 1);
    }
    for (int i = 0; i < U; ++i) {
      tc::mbar_init(sf_full + i, rank == 0 ? 5 : 4);
      tc::mbar_init(sf_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(acc_full + i, 1);
      tc::mbar_init(acc_empty + i, rank == 0 ? 5 : 4);
    }
    tc::mbar_init(done, 1);
    *abort_flag = 0;
    *no_flag = 0;
    tc::mbar_fence_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync();  // both blocks' barriers are there, and their tensor memory
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_previous(p.a_scales, p.w_scales, p.bias, p.Y);

  if (warp == 0) {
    // ------------------------------------------------------- code tiles
    if (lane == 0) {
      tc::tma_prefetch_map(&map_w);
      tc::tma_prefetch_map(&map_a);
      uint32_t it = 0;
      bool ok = true;
      for (int t = first; ok && t < p.tiles; t += stride) {
        const int f0 = (t % p.ftiles * 2 + rank) * kTF, m0 = t / p.ftiles * TN + rank * (TN / 2);
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const int s = it % S;
          ok = tc::mbar_wait(empty + s, (it / S & 1) ^ 1, abort_flag, p.status);
          if (!ok) break;
          const uint32_t dst = tc::smem_u32(codes_s + s * T::kCodes), bar = leader_address(codes_full + s);
          if (rank == 0) tc::mbar_arrive_expect_tx(codes_full + s, 2 * T::kCodes);
          tma_load_pair(dst, &map_w, kb * (kKB / 2), f0, bar);
          tma_load_pair(dst + T::kCodesF, &map_a, kb * (kKB / 2), m0, bar);
        }
      }
      // The blocks' memory outlives their copies, also after an abort (both blocks meet below).
      if (rank == 0)
        for (uint32_t i = it > S ? it - S : 0; i < it; ++i) tc::mbar_wait(codes_full + i % S, i / S & 1, no_flag, p.status);
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    // -------------------------------------------------------------- MMAs
    const bool leader = tc::elect_one();
    uint32_t it = 0, un = 0, n = 0;
    bool ok = true;
    for (int t = first; ok && t < p.tiles; t += stride, ++n) {
      const uint32_t buf = n & 1, acc = tmem + buf * TN;
      ok = wait_cluster(acc_empty + buf, (n >> 1 & 1) ^ 1, abort_flag, p.status);
      for (int kb = 0; ok && kb < p.kblocks; ++kb, ++it) {
        const int s = it % S, u = un % U, h = kb & 1;  // a unit's two stages
        if (h == 0) ok = wait_cluster(sf_full + u, un / U & 1, abort_flag, p.status);
        ok = ok && tc::mbar_wait_warp(codes_full + s, it / S & 1, abort_flag, p.status);
        // the MMAs that read this stage's scale slot before (with a slot per stage they are known to be done)
        if (T::kSfSlots < S && ok && it >= T::kSfSlots) {
          const uint32_t back = it - T::kSfSlots;
          ok = tc::mbar_wait_warp(empty + back % S, back / S & 1, abort_flag, p.status);
        }
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t wf = tc::smem_u32(codes_s + s * T::kCodes), tk = wf + T::kCodesF;
        const uint32_t sf = tc::smem_u32(sf_s + (u * 2 + h) * T::kSf);
        const uint32_t tf = tmem + 2 * TN + it % T::kSfSlots * T::kSfCols, tt = tf + 8;
        const bool last = kb + 1 == p.kblocks;
        if (leader) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            copy_scales_pair(tf + i * 4, sf + i * 512);
#pragma unroll
            for (int b = 0; b < T::kTokBlocks; ++b)
              copy_scales_pair(tt + (i * T::kTokBlocks + b) * 4, sf + T::kSfF + (i * T::kTokBlocks + b) * 512);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_mxf4_pair(acc, tc::desc_kmajor(wf, 0, k), tc::desc_kmajor(tk, 0, k), idesc_mxf4(2 * kTF, TN, (k & 1) * 2),
                          tf + (k >> 1) * 4, tt + (k >> 1) * T::kTokBlocks * 4, (kb | k) ? 1u : 0u);
          commit_pair(empty + s);
          if (h == 1 || last) commit_pair(sf_empty + u);
          if (last) commit_pair(acc_full + buf);
        }
        if (h == 1 || last) ++un;
        __syncwarp();
      }
    }
    if (leader) commit_pair(done);
    __syncwarp();
  } else if (warp == 1) {
    // Odd block: the word that an accumulator has been read.
    uint32_t n = 0;
    bool ok = true;
    for (int t = first; ok && t < p.tiles; t += stride, ++n) {
      ok = tc::mbar_wait_warp(acc_empty + (n & 1), n >> 1 & 1, abort_flag, p.status);
      if (ok && lane == 0) arrive_leader(acc_empty + (n & 1));
      __syncwarp();
    }
  } else if ((warp == 2 || warp == 3) && rank == 1) {
    // Every other unit each.
    const int units = (p.kblocks + 1) / 2;
    uint32_t un = 0;
    bool ok = true;
    for (int t = first; ok && t < p.tiles; t += stride)
      for (int i = 0; ok && i < units; ++i, ++un) {
        if ((un & 1) != (warp & 1)) continue;
        ok = tc::mbar_wait_warp(sf_full + un % U, un / U & 1, abort_flag, p.status);
        if (ok && lane == 0) arrive_leader(sf_full + un % U);
        __syncwarp();
      }
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ scales
    // Row r of the block's features and rows r, r + 128 of the tokens, loaded two
    // units ahead of the stores, over tile boundaries too.
    const int r = scale_row(threadIdx.x - 128);
    const int pitch = p.K / 32, units = (p.kblocks + 1) / 2;
    constexpr int R = T::kTokBlocks;
    struct Unit {
      uint4 v[R + 1];
    };
    int ft = first, fu = 0;  // the next unit to load
    auto fetch = [&](Unit& x) {
      const int f = (ft % p.ftiles * 2 + rank) * kTF + r, m0 = ft / p.ftiles * TN;
      const bool more = ft < p.tiles;
      x.v[0] = more && f < p.N ? load_scales(p.w_scales + (size_t)f * pitch, pitch, fu) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int b = 0; b < R; ++b) {
        const int m = r + b * 128;
        const bool there = more && m < TN && m0 + m < p.M;
        x.v[b + 1] = there ? load_scales(p.a_scales + (size_t)(m0 + m) * pitch, pitch, fu) : make_uint4(0, 0, 0, 0);
      }
      if (++fu == units) {
        fu = 0;
        ft += stride;
      }
    };
    Unit x0, x1, x2;
    fetch(x0);
    fetch(x1);
    uint32_t un = 0;
    bool ok = true;
    for (int t = first; ok && t < p.tiles; t += stride)
      for (int i = 0; i < units; ++i, ++un) {
        fetch(x2);
        ok = tc::mbar_wait_warp(sf_empty + un % U, (un / U & 1) ^ 1, abort_flag, p.status);
        if (!ok) break;
        // the four words of a row: stage 0 atoms 0, 1, stage 1 atoms 0, 1
        uint8_t* sf = sf_s + un % U * 2 * T::kSf + (threadIdx.x - 128) * 4;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint8_t* at = sf + (q >> 1) * T::kSf;
          auto word = [&](const uint4& v) { return q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w; };
          *reinterpret_cast<uint32_t*>(at + (q & 1) * 512) = word(x0.v[0]);
#pragma unroll
          for (int b = 0; b < R; ++b) *reinterpret_cast<uint32_t*>(at + T::kSfF + ((q & 1) * R + b) * 512) = word(x0.v[b + 1]);
        }
        tc::fence_proxy_async();  // the tensor core's copies read what this thread stored
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(sf_full + un % U);
        x0 = x1;
        x1 = x2;
      }
  } else if (warp >= 8) {
    // ---------------------------------------------------------- epilogue
    const int quarter = warp & 3, f = quarter * 32 + lane, tid = threadIdx.x - 256;
    uint32_t n = 0, step = 0;
    for (int t = first; t < p.tiles; t += stride, ++n) {
      const int f0 = (t % p.ftiles * 2 + rank) * kTF, m0 = t / p.ftiles * TN;
      const uint32_t buf = n & 1;
      const float bias = p.bias && f0 + f < p.N ? p.bias[f0 + f] : 0.f;
      if (!tc::bar_and(1, 128, tc::mbar_wait_warp(acc_full + buf, n >> 1 & 1, abort_flag, p.status))) break;
      tc::tc_fence_after();
      const int rows = min(TN, p.M - m0);
      for (int c = 0; c < rows; c += kChunk, ++step) {
        uint32_t v[32];
        tc::tmem_ld32(tc::taddr(tmem, quarter * 32, buf * TN + c), v);
        tc::tmem_ld_wait();
        bf16* st = out_s + (step & 1) * (kChunk * kTF);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) st[i * kTF + f] = __float2bfloat16_rn(__uint_as_float(v[i]) + bias);
        asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
        for (int u = 0; u < kChunk / 8; ++u) {
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
  }
  __syncthreads();
  cluster_sync();  // neither block's memory is in use by the other any more
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// ------------------------------------------------------------- few tokens
//
// Up to 64 tokens (and somewhat beyond, with few features and a long K) the
// product is a stream of the weights.  A cluster of C blocks shares a tile of 128
// features: block r takes the r-th part of K, and the partial sums meet through
// distributed shared memory, added in rank order (no workspace, no atomics, the
// same bits every time).  C grows while the blocks stay at about one per SM and
// each has two stages: a second wave costs more than the split gains (us, one
// token, K = 5,120, C = 1 / 2 / 4 / 8: N = 5,120 11.3 / 8.7 / 8.7 / 12.2; N =
// 15,360 12.2 / 12.6 / 16.6 / 25.5).

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

// Scales [8 kb, 8 kb + 8) of a row with `pitch` scales (one stage); 0 behind the end.
__device__ __forceinline__ uint2 load_scales8(const uint8_t* row, int pitch, int kb) {
  const uint8_t* s = row + kb * 8;
  if ((pitch & 7) == 0) return *reinterpret_cast<const uint2*>(s);
  const int left = pitch - kb * 8;
  uint32_t v[2] = {0, 0};
  if ((pitch & 3) == 0) {
    v[0] = *reinterpret_cast<const uint32_t*>(s);
    if (left > 4) v[1] = reinterpret_cast<const uint32_t*>(s)[1];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) v[i >> 2] |= (uint32_t)s[i] << (8 * (i & 3));
  }
  return make_uint2(v[0], v[1]);
}

template <int TN>
__global__ void __launch_bounds__(kFewThreads, 2)
    k_mx_few(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a, const ProductArgs args, int C) {
  using T = FewTile<TN>;
  constexpr int S = T::kStages;
  ProductArgs p = args;
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
  wait_previous(p.a_scales, p.w_scales, p.bias, p.Y);

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
          mma_mxf4(tmem, tc::desc_kmajor(wf, 0, k), tc::desc_kmajor(tk, 0, k), idesc_mxf4(kTF, TN, (k & 1) * 2), tf + (k >> 1) * 4,
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
    const int r = scale_row(threadIdx.x - 128), pitch = p.K / 32;
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
        uint8_t* sf = sf_s + s * T::kSf + (threadIdx.x - 128) * 4;
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
          else if (c + i < rows && f0 + f < p.N)
            p.Y[(size_t)(m0 + c + i) * p.N + f0 + f] = __float2bfloat16_rn(__uint_as_float(v[i]) + bias);
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

// Blocks that share a tile of 128 features x TN tokens in k_mx_few.
int few_split(int tiles, int kblocks) {
  int C = 1;
  while (C < 8 && tiles * C * 2 <= 160 && kblocks >= 4 * C) C *= 2;
  return C;
}
int few_tiles(int M, int N, int TN) { return (int)std::min(1LL << 30, (long long)((N + kTF - 1) / kTF) * ((M + TN - 1) / TN)); }

template <int TN>
cudaError_t launch_few(ProductArgs p, const uint8_t* a_codes, const uint8_t* w_codes, cudaStream_t st) {
  using T = FewTile<TN>;
  CUtensorMap map_w, map_a;
  if (!tma_map_u8_rows(&map_w, w_codes, p.K / 2, p.N, kTF) || !tma_map_u8_rows(&map_a, a_codes, p.K / 2, p.M, TN))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_dynamic_smem(k_mx_few<TN>, T::kSmem);
  if (e != cudaSuccess) return e;
  p.ftiles = (p.N + kTF - 1) / kTF;
  p.tiles = few_tiles(p.M, p.N, TN);
  const int C = few_split(p.tiles, p.kblocks);
  note_launch();
  return launch_chained(k_mx_few<TN>, p.tiles * C, kFewThreads, T::kSmem, C, st, map_w, map_a, p, C);
}

template <int TN>
cudaError_t launch_pair(ProductArgs p, const uint8_t* a_codes, const uint8_t* w_codes, cudaStream_t st) {
  using T = Pair<TN>;
  CUtensorMap map_w, map_a;
  if (!tma_map_u8_rows(&map_w, w_codes, p.K / 2, p.N, kTF) || !tma_map_u8_rows(&map_a, a_codes, p.K / 2, p.M, TN / 2))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_dynamic_smem(k_mx_pair<TN>, T::kSmem);
  if (e != cudaSuccess) return e;
  p.ftiles = (p.N + 2 * kTF - 1) / (2 * kTF);
  p.tiles = p.ftiles * ((p.M + TN - 1) / TN);
  note_launch();
  return launch_chained(k_mx_pair<TN>, 2 * std::min(p.tiles, 74), kPairThreads, T::kSmem, 0, st, map_w, map_a, p);
}

// Relative time of a product in tiles of TN tokens: the rounds of tiles that 74
// pairs of SMs take, times what a round takes (2,048 x 15,360 x 5,120, us for a
// round of 64 / 128 / 192: 6.0 / 7.5 / 8.7; one of 224 takes 1.04 to 1.13 times
// one of 192, since its scales wait).
long long pair_cost(int M, int N, int TN) {
  const long long tiles = (long long)((N + 2 * kTF - 1) / (2 * kTF)) * ((M + TN - 1) / TN);
  return (tiles + 73) / 74 * (TN + (TN > 192 ? 256 : 237));
}

}  // namespace

cudaError_t mx_product_run(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* w_codes, const uint8_t* w_scales,
                           const float* bias, int M, int N, int K, void* Y, cudaStream_t st) {
  ProductArgs p{};
  p.a_scales = a_scales; p.w_scales = w_scales; p.bias = bias;
  p.Y = static_cast<bf16*>(Y);
  p.M = M; p.N = N; p.K = K;
  p.kblocks = (K + kKB - 1) / kKB;
  p.status = status_word();
  if (!p.status) return cudaErrorInvalidValue;
  if (M <= 16) return launch_few<16>(p, a_codes, w_codes, st);
  // Beyond 64 tokens a long K that four blocks or more would share is still theirs
  // (us, this / pairs: 128 x 2,048 x 8,192 9.6 / 15.3; 512 x 512 x 8,192 9.6 /
  // 13.8; with two blocks 300 x 2,048 x 8,192 15.5 / 15.3, with one 512 x 2,048 x
  // 8,192 17.8 / 15.5).
  if (M <= 64 || few_split(few_tiles(M, N, 64), p.kblocks) >= 4) return launch_few<64>(p, a_codes, w_codes, st);
  // The width whose rounds take the least (us for 64 / 128 / 192 / 224 tokens:
  // 512 x 2,048 x 2,048 7.9 / 8.4 / 9.3 / 10.1; 2,048 x 2,048 x 2,048 14.7 / 11.1
  // / 12.0 / 11.9; 512 x 5,120 x 5,120 22.8 / 18.5 / 14.7 / 16.0; 1,500 x 5,120 x
  // 5,120 45.4 / 30.7 / 27.7 / 24.3; 75,600 x 15,360 x 5,120 at 192 / 224 2,720 /
  // 2,530).
  int best = 64;
  for (const int tn : {128, 192, 224})
    if (pair_cost(M, N, tn) <= pair_cost(M, N, best)) best = tn;
  if (best == 64) return launch_pair<64>(p, a_codes, w_codes, st);
  if (best == 128) return launch_pair<128>(p, a_codes, w_codes, st);
  if (best == 192) return launch_pair<192>(p, a_codes, w_codes, st);
  return launch_pair<224>(p, a_codes, w_codes, st);
}

}  // namespace svg
