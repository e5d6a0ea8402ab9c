// Device code shared by the four-bit products: block-scaled MMAs and the copies
// of scales into tensor memory.
#pragma once
#include "fp4_kernels.h"
#include "gemm_common.cuh"

namespace tpmlp {
namespace fp4 {

// A k-tile is 256 elements, 128 bytes of codes: four MMAs of K = 64.
constexpr int KSTEPS = 4;

// Scales in tensor memory: of a 128-row operand tile, row r's four bytes lie in
// lane r mod 32 (and again in lanes + 32, + 64, + 96) of column r / 32.  One
// copy moves the 512 bytes that hold four blocks of 128 rows into 4 columns.
// NV: four blocks are one K step (64 elements, scale_vec::4X).  MX: two K steps,
// the first reads bytes 0 and 1, the second 2 and 3 (scale_vec::2X).
__host__ __device__ constexpr int copies_per_tile(int format) {
  return format == TPFP4_NV ? 4 : 2;
}

// Shared-memory descriptor of those 512 bytes: no swizzle, groups of 8 rows of
// 16 bytes, 128 bytes apart.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) |
         (static_cast<uint64_t>(128 >> 4) << 32) | (1ull << 46);
}

__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr),
               "l"(desc)
               : "memory");
}
// Both CTAs of the pair, each from its own shared memory.
__device__ __forceinline__ void copy_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr),
               "l"(desc)
               : "memory");
}

// Instruction descriptor of the block-scaled kinds: A and B E2M1 (format 1 in
// bits 7-9 and 10-12), N >> 3 (bits 17-22), scale type (bit 23: 0 E4M3, 1
// E8M0), M >> 4 (bits 24-28), the scales' byte offset of A (bits 29-30) and B
// (bits 4-5); K-major, K = 64.
__host__ __device__ constexpr uint32_t idesc_fp4(int format, int M, int N,
                                                 int byte) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         ((format == TPFP4_MX ? 1u : 0u) << 23) |
         (static_cast<uint32_t>(M >> 4) << 24) |
         (static_cast<uint32_t>(byte) << 29) | (static_cast<uint32_t>(byte) << 4);
}

template <int FORMAT, int CTAS>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b,
                                        uint32_t idesc, uint32_t sa, uint32_t sb,
                                        uint32_t accumulate) {
#define TPMLP_MMA_FP4(group, kind, vec)                                      \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"             \
               "tcgen05.mma.cta_group::" group ".kind::" kind                \
               ".block_scale.scale_vec::" vec                                \
               " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),            \
               "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate) \
               : "memory")
  if constexpr (FORMAT == TPFP4_NV) {
    if constexpr (CTAS == 2)
      TPMLP_MMA_FP4("2", "mxf4nvf4", "4X");
    else
      TPMLP_MMA_FP4("1", "mxf4nvf4", "4X");
  } else {
    if constexpr (CTAS == 2)
      TPMLP_MMA_FP4("2", "mxf4", "2X");
    else
      TPMLP_MMA_FP4("1", "mxf4", "2X");
  }
#undef TPMLP_MMA_FP4
}

// One lane of a converged warp, the same one every time (commits cover what
// their own thread issued).  The loops around it are the whole warp's: the
// compiler then keeps descriptors and addresses in uniform registers, where
// these instructions take them.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
               "selp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(yes));
  return yes != 0;
}

// Arrive on a barrier of the pair's other CTA, for tensor memory that has been
// read: no memory of this thread's is handed over, so the arrival does not wait
// for its earlier stores (a release at cluster scope did, 1600 cycles a tile).
__device__ __forceinline__ void arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                   cluster_addr)
               : "memory");
}

// The whole warp's bounded wait (see gemm::wait_bounded): whether the phase
// completed.  (A try suspends for 10 to 20 us, so that budgets below that are
// those; spinning on test_wait instead: 8192 x 5120 x 20480 250 us, not 241.)
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity,
                                          const gemm::Ctl& c, int role) {
  if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (true) {
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *c.abort_flag != 0)) return false;
    if (!__any_sync(0xffffffffu, ptx::globaltimer_ns() - t0 > c.budget)) continue;
    if ((threadIdx.x & 31) == 0) {
      *c.abort_flag = 1;
      if (atomicCAS(c.status, 0, TPMLP_ERR_TIMEOUT) == 0) {
        c.status[1] = role;
        c.status[2] = static_cast<int>(blockIdx.x);
      }
      __threadfence();
    }
    __syncwarp();
    return false;
  }
}

// One k-tile: its scales into tensor memory (columns t_sa and t_sb on), then
// its four MMAs.  A copy and the MMAs issued after it, and MMAs and the copies
// after them, run in the order of issue.  a, b: descriptors of the operands'
// tiles, sa, sb: of their scale tiles; SB_TILES: 128-row tiles of B's scales.
template <int FORMAT, int CTAS, int M, int N, int SB_TILES>
__device__ __forceinline__ void ktile_mmas(uint32_t d, uint64_t a, uint64_t b,
                                           uint64_t sa, uint64_t sb,
                                           uint32_t t_sa, uint32_t t_sb,
                                           bool first) {
  constexpr int COPIES = copies_per_tile(FORMAT);
  constexpr int TILE = tile_bytes(FORMAT);
#pragma unroll
  for (int i = 0; i < COPIES; ++i) {
    if constexpr (CTAS == 2)
      copy_scales_pair(t_sa + 4 * i, sa + i * 512 / 16);
    else
      copy_scales(t_sa + 4 * i, sa + i * 512 / 16);
#pragma unroll
    for (int j = 0; j < SB_TILES; ++j) {
      if constexpr (CTAS == 2)
        copy_scales_pair(t_sb + 4 * (i * SB_TILES + j),
                         sb + (j * TILE + i * 512) / 16);
      else
        copy_scales(t_sb + 4 * (i * SB_TILES + j), sb + (j * TILE + i * 512) / 16);
    }
  }
#pragma unroll
  for (int k = 0; k < KSTEPS; ++k) {
    const int copy = k * COPIES / KSTEPS;
    const uint32_t idesc =
        FORMAT == TPFP4_NV
            ? idesc_fp4(FORMAT, M, N, 0)
            : (k % 2 ? idesc_fp4(FORMAT, M, N, 2) : idesc_fp4(FORMAT, M, N, 0));
    mma_fp4<FORMAT, CTAS>(d, a + k * 32 / 16, b + k * 32 / 16, idesc,
                          t_sa + 4 * copy, t_sb + 4 * SB_TILES * copy,
                          first && k == 0 ? 0u : 1u);
  }
}

}  // namespace fp4
}  // namespace tpmlp
