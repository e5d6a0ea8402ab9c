// The four-bit product on CTA pairs: C = g_A g_B A B^T with A [M, K] and
// B [N, K] packed (E2M1 codes, a scale for 16 or 32 elements of K), 256 x 256
// output tiles, persistent.
//
// The tensor cores take the scales with the operands (tcgen05.mma .block_scale):
// an MMA of K = 64 reads 32 bytes of codes a row and its 4 (NV) or 2 (MX) scale
// bytes a row from tensor memory, where tcgen05.cp puts them; the matrices'
// layout of scales is the one that copy reads, so that they go from global to
// tensor memory untouched.  Per k-tile (256 elements) a CTA loads its 128 rows
// of A and of B (16 KB each), its own rows' scales (2 KB, NV) and the scales of
// all 256 rows of B (4 KB): each SM multiplies its A rows with the B columns
// of both.
//
// 12 warps: warp 0 loads, warp 1 of the even CTA copies scales and issues the
// MMAs (one elected lane each), warps 4-11 are the epilogue: warp w takes TMEM
// lanes 32 (w mod 4) on and one 128-column half.
//
// Tensor memory: two accumulators of 256 columns would fill all 512, and the
// scales need 48.  So the second one starts at column 208, over the last 48 of
// the first: the MMAs of tile j + 1 may start once tile j's part of the shared
// 48 columns has been read, which the warps that own them do first.
//
//   full[s]   (even CTA) bytes of stage s landed in both CTAs
//   empty[s]  (each CTA) the MMAs have read stage s
//   tfull     (each CTA) tile j's accumulator is ready
//   shared    (even CTA) 16 arrivals, one a warp of the pair: it has read all of
//             tile j - 1 and its part of tile j's shared columns.
// Every wait is bounded, as in gemm_tc2.cu: on expiry TPMLP_ERR_TIMEOUT goes to
// the status word, the roles stop and tensor memory is freed.
//
// Measured: 8192 x 15360 x 5120 187 us NV (6.9 PFLOP/s), 180 MX; 8192 x 5120 x 20480
// 236 NV (7.3 PFLOP/s), 222 MX (7.7).  A k-tile's MMAs take 512 cycles.  With 12
// pairs it takes 591, with all 76 690 at 2070 MHz (operands of zeros: no power cap;
// 17 TB/s out of L2).  Operands of random values run into the power cap: at 1.6 GHz,
// after seconds of them, 622 cycles.  What holds the cycles past 512 is not shown: the
// profiler has the tensor pipe as the busiest unit (67 % of a launch of 8.4 rounds), L2
// at 47 % and L1 and shared memory at 41 %; one write and one read of a stage's 38912
// bytes (NV) at 128 bytes a cycle would be 608 cycles if the two excluded one another,
// more than the 591 measured.  256 x 256 is the largest tile whose accumulators leave
// tensor memory for the scales.
#include <climits>

#include "fp4_gemm.cuh"
#include "host_common.cuh"

namespace tpmlp {
namespace fp4 {
namespace {

using namespace gemm;

constexpr int PM = 256, PN = 256;   // a pair's tile
constexpr int HM = 128;             // rows of A a CTA loads
constexpr int STAGES = 5;
constexpr int NUM_THREADS = 384;
constexpr int NUM_EPI_WARPS = 8;
constexpr int FIRST_EPI_WARP = 4;
constexpr int REGS_LAUNCH = 168;
constexpr int REGS_CONTROL = 56;
constexpr int REGS_EPILOGUE = 224;
static_assert(REGS_CONTROL * 128 + REGS_EPILOGUE * 256 <=
                  REGS_LAUNCH * NUM_THREADS,
              "register split exceeds the launch allocation");
constexpr uint32_t OPERAND_BYTES = HM * 128;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t ACC_STEP = 208;   // the second accumulator's first column
constexpr uint32_t T_SA = 464, T_SB = 480;
constexpr int NUM_BARRIERS = 2 * STAGES + 3;   // full, empty, tfull, shared, done
constexpr uint32_t STAGING_BYTES = NUM_EPI_WARPS * STAGE_CHUNK_BYTES;
// Rows of tiles that are walked together: 8192 x 20480 x 5120 takes 255 us with
// 8, 247 with 16, 8192 x 5120 x 20480 237 and 239.
constexpr int GROUP_M = 16;
constexpr unsigned long long ABORT_SETTLE_NS = 2000000ull;

template <int FORMAT>
constexpr uint32_t stage_bytes() {
  return 2 * OPERAND_BYTES + 3 * tile_bytes(FORMAT);
}
template <int FORMAT>
constexpr size_t smem_bytes() {
  return 1024 + size_t(STAGES) * stage_bytes<FORMAT>() + STAGING_BYTES +
         NUM_BARRIERS * 8 + 16;
}
static_assert(smem_bytes<TPFP4_NV>() <= 227 * 1024, "shared memory budget");

__device__ __forceinline__ void cta_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(NUM_THREADS) : "memory");
}

// A unit of a pair's work: a tile, or 128 of its columns.  Where a last round of
// tiles would leave half the pairs idle or more, its tiles are dealt out as
// halves (8192 x 5120 x 5120: 640 tiles, 8.42 rounds of 76, 66.5 us instead of 68.1;
// 512 x 4096 x 4096: 32 tiles, 8.3 instead of 9.2).
struct Item {
  int m0, n0;    // the pair's first row and column
  int cols;      // 256 or 128; 0: a half that lies past the matrix
};
template <int EPI>
__device__ __forceinline__ Item item_of(int item, int whole, int num_m, int num_n,
                                        int group_m, int N) {
  const int half = item - whole;
  int mb, nb;
  tile_coords(half < 0 ? item : whole + half / 2, num_m, num_n, group_m, mb, nb);
  Item it;
  it.m0 = mb * PM;
  it.n0 = nb * PN + (half < 0 ? 0 : half % 2 * (PN / 2));
  // (OUT_GELU_FP4 writes what its output's last k-tile holds past the matrix)
  it.cols = half < 0 ? PN : it.n0 < N || EPI == OUT_GELU_FP4 ? PN / 2 : 0;
  return it;
}

// bias[c0 .. c0 + 64) of which n are in the matrix.
__device__ __forceinline__ void add_bias(const float* bias, int c0, int n,
                                         float (&v)[64]) {
  if (bias == nullptr) return;
  if (n >= 64 && (reinterpret_cast<uintptr_t>(bias) & 15u) == 0) {
#pragma unroll
    for (int i = 0; i < 64; i += 4) {
      const uint4 u = load_u32x4(bias + c0 + i);
      v[i] += __uint_as_float(u.x);
      v[i + 1] += __uint_as_float(u.y);
      v[i + 2] += __uint_as_float(u.z);
      v[i + 3] += __uint_as_float(u.w);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 64; ++i)
    if (i < n) v[i] += load_f32(bias + c0 + i);
}

// One warp's staging buffer: 32 rows of 128 bytes (16-byte unit u of row r at
// unit u ^ r mod 8), written out by TMA, or, where the output's rows are not
// 16-byte aligned, by the warp, row by row (8192 x 5120 x 5120: 66 and 71 us).
struct Stager {
  uint32_t buf;
  int lane;

  __device__ __forceinline__ void write(const uint32_t* w) {
    const uint32_t row = buf + static_cast<uint32_t>(lane) * 128u;
#pragma unroll
    for (int c = 0; c < 8; ++c)
      ptx::st_shared_v4(row + static_cast<uint32_t>(c ^ (lane & 7)) * 16u,
                        w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  }
  __device__ __forceinline__ void put_tma(const CUtensorMap* map, int c0, int r0,
                                          const uint32_t* w) {
    if (lane == 0) ptx::bulk_wait_read<0>();
    __syncwarp();
    write(w);
    ptx::fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
      ptx::tma_store_2d(map, buf, c0, r0);
      ptx::bulk_commit();
    }
  }
  // rows and cols: what of the chunk is in the matrix
  template <bool F32>
  __device__ __forceinline__ void put_rows(void* out, long long ld, int c0, int r0,
                                           int rows, int cols, const uint32_t* w) {
    __syncwarp();
    write(w);
    __syncwarp();
    for (int r = 0; r < min(rows, 32); ++r) {
      const uint32_t word = ptx::ld_shared_u32(
          buf + static_cast<uint32_t>(r) * 128u +
          static_cast<uint32_t>((lane >> 2) ^ (r & 7)) * 16u + (lane & 3) * 4u);
      if constexpr (F32) {
        if (lane < cols)
          static_cast<float*>(out)[(r0 + r) * ld + c0 + lane] =
              __uint_as_float(word);
      } else {
        auto* p = static_cast<unsigned short*>(out) + (r0 + r) * ld + c0 + 2 * lane;
        if (2 * lane < cols) p[0] = static_cast<unsigned short>(word);
        if (2 * lane + 1 < cols) p[1] = static_cast<unsigned short>(word >> 16);
      }
    }
  }
  __device__ __forceinline__ void drain() {
    if (lane == 0) ptx::bulk_wait_all();
    __syncwarp();
  }
};

// 64 columns of a row, GeLU taken, quantised and stored.
template <int FORMAT>
__device__ __forceinline__ void store_fp4(const Packed& y, int row, int c0,
                                          float inv_g, const float (&v)[64]) {
  constexpr int BLOCK = block_size(FORMAT);
  constexpr int BLOCKS = 64 / BLOCK;
  uint32_t word = 0, c[8];
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < BLOCK; ++i) amax = max(amax, abs_bits(v[b * BLOCK + i]));
    const Scale s = block_scale<FORMAT>(amax, inv_g);
    word |= s.byte << (8 * b);
#pragma unroll
    for (int i = 0; i < BLOCK / 16; ++i) {
      const uint2 w = codes16<FORMAT, true>(v + b * BLOCK + 16 * i, s);
      c[b * BLOCK / 8 + 2 * i] = w.x;
      c[b * BLOCK / 8 + 2 * i + 1] = w.y;
    }
  }
  uint8_t* dst = y.codes + code_row(row, c0 / TILE_COLS, y.ktiles);
  const int unit = c0 % TILE_COLS / 32;
  *reinterpret_cast<uint4*>(dst + code_unit(row, unit)) =
      make_uint4(c[0], c[1], c[2], c[3]);
  *reinterpret_cast<uint4*>(dst + code_unit(row, unit + 1)) =
      make_uint4(c[4], c[5], c[6], c[7]);
  const int block = c0 % TILE_COLS / BLOCK;
  uint8_t* to = y.scales + scale_word(row, c0 / TILE_COLS, block / 4, y.ktiles,
                                      tile_bytes(FORMAT)) + block % 4;
  if constexpr (FORMAT == TPFP4_NV)
    *reinterpret_cast<uint32_t*>(to) = word;
  else
    *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(word);
}

// 64 columns past the matrix in its last k-tile, which its products read.
template <int FORMAT>
__device__ __forceinline__ void store_nothing(const Packed& y, int row, int c0) {
  uint8_t* dst = y.codes + code_row(row, c0 / TILE_COLS, y.ktiles);
  const int unit = c0 % TILE_COLS / 32;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    *reinterpret_cast<uint4*>(dst + code_unit(row, unit + i)) =
        make_uint4(0u, 0u, 0u, 0u);
  const int block = c0 % TILE_COLS / block_size(FORMAT);
  uint8_t* to = y.scales + scale_word(row, c0 / TILE_COLS, block / 4, y.ktiles,
                                      tile_bytes(FORMAT)) + block % 4;
  if constexpr (FORMAT == TPFP4_NV)
    *reinterpret_cast<uint32_t*>(to) = 0u;
  else
    *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(0x7f7fu);
}

template <int FORMAT, int EPI>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    product_pairs_kernel(const __grid_constant__ CUtensorMap tmA,
                         const __grid_constant__ CUtensorMap tmSA,
                         const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmSB,
                         const __grid_constant__ CUtensorMap tmO,
                         const ProductArgs args, const int tma_out,
                         const int group_m, const int halves) {
  constexpr uint32_t TILE = tile_bytes(FORMAT);
  constexpr uint32_t STAGE = stage_bytes<FORMAT>();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s_a = ptx::smem_u32(smem);
  const uint32_t s_b = s_a + STAGES * OPERAND_BYTES;
  const uint32_t s_epi = s_b + STAGES * OPERAND_BYTES;
  const uint32_t s_sa = s_epi + STAGING_BYTES;
  const uint32_t s_sb = s_sa + STAGES * TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + size_t(STAGES) * STAGE +
                                               STAGING_BYTES);
  const uint32_t full0 = ptx::smem_u32(bars);
  const uint32_t empty0 = full0 + 8u * STAGES;
  const uint32_t tfull = empty0 + 8u * STAGES;
  const uint32_t shared = tfull + 8u;
  const uint32_t done_bar = shared + 8u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NUM_BARRIERS);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  if (args.dependent) let_next_launch_start();
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t prank = ptx::cluster_ctarank();
  const bool leader = prank == 0;
  const int pair = static_cast<int>(blockIdx.x >> 1);
  const int num_pairs = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(full0 + 8u * s, 1);
      ptx::mbar_init(empty0 + 8u * s, 1);
    }
    ptx::mbar_init(tfull, 1);
    ptx::mbar_init(shared, 2 * NUM_EPI_WARPS);
    ptx::mbar_init(done_bar, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmSA);
    ptx::prefetch_tmap(&tmB);
    ptx::prefetch_tmap(&tmSB);
    if (EPI != OUT_GELU_FP4 && tma_out) ptx::prefetch_tmap(&tmO);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), TMEM_COLS);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();   // barriers of both CTAs initialised, TMEM allocated
  ptx::tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);

  if (!args.dependent) {
    wait_for_launch_before();
    let_next_launch_start();
  }
  const Ctl ctl{abort_flag, args.status, args.budget_ns};
  const int num_m = (args.M + PM - 1) / PM;
  const int num_n = (args.N + PN - 1) / PN;
  const int whole = num_m * num_n - halves;   // tiles dealt out whole
  const int items = whole + 2 * halves;
  const int ktiles = args.a.ktiles;
  const uint32_t lead_full0 = ptx::mapa_shared(full0, 0u);
  const uint32_t lead_shared = ptx::mapa_shared(shared, 0u);

  if (warp < FIRST_EPI_WARP) {
    ptx::setmaxnreg_dec<REGS_CONTROL>();
    if (warp == 0) {
      // ---------------------------------------------------- producer --
      uint32_t stage = 0, phase = 0;
      bool alive = true;
      for (int item = pair; alive && item < items; item += num_pairs) {
        const Item it = item_of<EPI>(item, whole, num_m, num_n, group_m, args.N);
        if (it.cols == 0) continue;
        // tile numbers; tiles past the matrix are filled with zeros.  B comes in
        // boxes of 64 rows: a CTA takes half of the item's columns.
        const int ta0 =
            (it.m0 / TILE_ROWS + static_cast<int>(prank)) * ktiles;
        const int n0 = it.n0 + static_cast<int>(prank) * it.cols / 2;
        const int tb0 = n0 / TILE_ROWS * ktiles, row0 = n0 % TILE_ROWS;
        const int sb0 = it.n0 / TILE_ROWS * ktiles;
        const bool full = it.cols == PN;
        const uint32_t bytes =
            full ? STAGE : OPERAND_BYTES + OPERAND_BYTES / 2 + 2 * TILE;
        auto load_b = [&](int kt, uint32_t st) {
          if (leader) ptx::mbar_arrive_expect_tx(full0 + 8u * st, 2 * bytes);
          const uint32_t fb = lead_full0 + 8u * st;
          const uint32_t db = s_b + st * OPERAND_BYTES;
          const int rb = (tb0 + kt) * TILE_ROWS + row0;
          ptx::tma_load_2d_pair(db, &tmB, fb, 0, rb);
          ptx::tma_load_2d_pair(s_sb + st * 2 * TILE, &tmSB, fb, 0, sb0 + kt);
          if (full) {
            ptx::tma_load_2d_pair(db + OPERAND_BYTES / 2, &tmB, fb, 0, rb + 64);
            ptx::tma_load_2d_pair(s_sb + st * 2 * TILE + TILE, &tmSB, fb, 0,
                                  sb0 + ktiles + kt);
          }
        };
        auto load_a = [&](int kt, uint32_t st) {
          const uint32_t fb = lead_full0 + 8u * st;
          ptx::tma_load_2d_pair(s_a + st * OPERAND_BYTES, &tmA, fb, 0,
                                (ta0 + kt) * TILE_ROWS);
          ptx::tma_load_2d_pair(s_sa + st * TILE, &tmSA, fb, 0, ta0 + kt);
        };
        int early = 0;   // k-tiles of B loaded before A may be read
        if (item == pair) {
          early = min(ktiles, STAGES);
          if (elect_one())
            for (int kt = 0; kt < early; ++kt) load_b(kt, kt);
          __syncwarp();
          wait_for_launch_before();
        }
        for (int kt = 0; kt < ktiles; ++kt) {
          if (!wait_warp(empty0 + 8u * stage, phase ^ 1u, ctl, ROLE_PRODUCER)) {
            alive = false;
            break;
          }
          if (elect_one()) {
            if (kt >= early) load_b(kt, stage);
            load_a(kt, stage);
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    } else if (warp == 1 && leader) {
      // -------------------------------------------------- MMA issuer --
      constexpr uint16_t pair_mask = 0x3;
      const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
      const uint64_t desc_a = ptx::sdesc_sw128(s_a, 16, 1024);
      const uint64_t desc_b = ptx::sdesc_sw128(s_b, 16, 1024);
      const uint64_t desc_sa = sdesc_scales(s_sa);
      const uint64_t desc_sb = sdesc_scales(s_sb);
      uint32_t stage = 0, phase = 0, j = 0;
      bool alive = true;
      wait_for_launch_before();   // not on a bounded wait's budget
      for (int item = pair; alive && item < items; item += num_pairs) {
        const Item it = item_of<EPI>(item, whole, num_m, num_n, group_m, args.N);
        if (it.cols == 0) continue;
        if (j > 0 && !wait_warp(shared, (j - 1u) & 1u, ctl, ROLE_MMA)) {
          alive = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t d = tmem + (j & 1u) * ACC_STEP;
        for (int kt = 0; kt < ktiles; ++kt) {
          if (!wait_warp(full0 + 8u * stage, phase, ctl, ROLE_MMA)) {
            alive = false;
            break;
          }
          ptx::tc_fence_after();
          if (elect_one()) {
            const uint64_t da = desc_a + stage * (OPERAND_BYTES / 16);
            const uint64_t db = desc_b + stage * (OPERAND_BYTES / 16);
            const uint64_t dsa = desc_sa + stage * (TILE / 16);
            const uint64_t dsb = desc_sb + stage * (2 * TILE / 16);
            if (it.cols == PN)
              ktile_mmas<FORMAT, 2, PM, PN, 2>(d, da, db, dsa, dsb, tmem + T_SA,
                                               tmem + T_SB, kt == 0);
            else
              ktile_mmas<FORMAT, 2, PM, PN / 2, 1>(d, da, db, dsa, dsb, tmem + T_SA,
                                                   tmem + T_SB, kt == 0);
            ptx::mma_commit_pair(empty0 + 8u * stage, pair_mask);
            if (kt == ktiles - 1) ptx::mma_commit_pair(tfull, pair_mask);
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        ++j;
      }
      if (*reinterpret_cast<volatile int*>(abort_flag)) {
        // Wait for every MMA issued before TMEM is freed.
        if (elect_one())
          ptx::mma_commit_pair(done_bar, static_cast<uint16_t>(1u << prank));
        __syncwarp();
        wait_teardown(done_bar, 0);
      }
    }
    // ------------------------------------------------------ teardown --
    cta_barrier();
    if (*reinterpret_cast<volatile int*>(abort_flag) && warp == 0 &&
        lane == 0) {
      // copies may still land here, counted on the peer's barrier
      const uint64_t t0 = ptx::globaltimer_ns();
      while (ptx::globaltimer_ns() - t0 < ABORT_SETTLE_NS) {
      }
    }
    cta_barrier();
    ptx::cluster_sync();
    if (warp == 1) {
      __syncwarp();
      ptx::tc_fence_after();
      ptx::tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
  } else {
    ptx::setmaxnreg_inc<REGS_EPILOGUE>();
    // ------------------------------------------------------ epilogue --
    const int ew = warp - FIRST_EPI_WARP;
    const int q = warp & 3;      // TMEM sub-partition this warp may read
    const int half = ew >> 2;    // which 128-column half of the tile
    Stager st{s_epi + static_cast<uint32_t>(ew) * STAGE_CHUNK_BYTES, lane};
    wait_for_launch_before();
    const float2 g = gain_factors(args.a.head->g, args.b.head->g);
    float inv_gy = 1.f;
    if constexpr (EPI == OUT_GELU_FP4) {
      inv_gy = exp2_of(-args.y_exponent);
      if (blockIdx.x == 0 && threadIdx.x == FIRST_EPI_WARP * 32) {
        args.y.head->g = exp2_of(args.y_exponent);
        for (int i = 0; i < 4; ++i) args.y.head->status[i] = 0;
      }
    }
    uint32_t j = 0;
    for (int item = pair; item < items; item += num_pairs) {
      const Item it = item_of<EPI>(item, whole, num_m, num_n, group_m, args.N);
      if (it.cols == 0) continue;
      const int row0 = it.m0 + static_cast<int>(prank) * HM + q * 32;
      const int row = row0 + lane;
      const int chunks = it.cols / 128;   // of 64 columns, this warp's
      if (!wait_warp(tfull, j & 1u, ctl, ROLE_EPILOGUE)) break;
      ptx::tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                             (j & 1u) * ACC_STEP;
      // the shared columns: of the first accumulator its last 48 (which a half
      // does not use), of the second its first
      const bool owner = (j & 1u) ? half == 0 : half == 1 && chunks == 2;
      ++j;
      auto release = [&] {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader)
            ptx::mbar_arrive(shared);
          else
            arrive_relaxed(lead_shared);
        }
      };
      if (!owner) release();
#pragma unroll 1
      for (int jj = 0; jj < chunks; ++jj) {
        const int chunk = owner && half == 1 ? 1 - jj : jj;
        const int col = (half * chunks + chunk) * 64;
        const int c0 = it.n0 + col;
        uint32_t r0[32], r1[32];
        ptx::tmem_ld_32x32b_x32(taddr + col, r0);
        ptx::tmem_ld_32x32b_x32(taddr + col + 32, r1);
        ptx::tmem_ld_wait();
        if (owner && jj == 0) release();
        if (row0 >= args.M) continue;
        if (c0 >= args.N) {
          if constexpr (EPI == OUT_GELU_FP4) {
            if (row < args.M && c0 < args.y.ktiles * TILE_COLS)
              store_nothing<FORMAT>(args.y, row, c0);
          }
          continue;
        }
        const int n = args.N - c0;
        float v[64];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          v[i] = __uint_as_float(r0[i]) * g.x;
          v[32 + i] = __uint_as_float(r1[i]) * g.x;
        }
        if (g.y != 1.f) {   // (always multiplied, 8192 x 5120 x 20480 takes 1 us more)
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i] *= g.y;
        }
        add_bias(args.bias, c0, n, v);
        if constexpr (EPI == OUT_GELU_FP4) {
#pragma unroll
          for (int i = 0; i < 64; i += 2)
            gelu2_f32(v[i], v[i + 1], args.gelu_mode);
          if (row < args.M) store_fp4<FORMAT>(args.y, row, c0, inv_gy, v);
        } else if constexpr (EPI == OUT_BF16) {
          add_residual_bf16(args.residual, args.ldr, row, args.M, c0, v, 64);
          uint32_t w[32];
          pack_bf16x64(v, w);
          if (tma_out)
            st.put_tma(&tmO, c0, row0, w);
          else
            st.put_rows<false>(args.out, args.ldo, c0, row0, args.M - row0, n, w);
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[32 * k + i]);
            if (n <= 32 * k) continue;
            if (tma_out)
              st.put_tma(&tmO, c0 + 32 * k, row0, w);
            else
              st.put_rows<true>(args.out, args.ldo, c0 + 32 * k, row0,
                                args.M - row0, n - 32 * k, w);
          }
        }
      }
    }
    st.drain();
    cta_barrier();
    cta_barrier();
    ptx::cluster_sync();
  }
}

template <int FORMAT, int EPI>
cudaError_t launch_pairs(const CUtensorMap& ta, const CUtensorMap& tsa,
                         const CUtensorMap& tb, const CUtensorMap& tsb,
                         const CUtensorMap* to, const ProductArgs& args,
                         int max_pairs, cudaStream_t s) {
  auto kern = product_pairs_kernel<FORMAT, EPI>;
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs * NUM_THREADS <
      REGS_CONTROL * 128 + REGS_EPILOGUE * NUM_EPI_WARPS * 32)
    return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem_bytes<FORMAT>()));
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>((args.M + PM - 1) / PM) *
                          ((args.N + PN - 1) / PN);
  if (tiles > INT_MAX / 2) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = smem_bytes<FORMAT>();
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const long long last = tiles % max_pairs;   // tiles of the last round
  const long long halves = 2 * last <= max_pairs ? last : 0;
  const long long items = tiles + halves;
  cfg.gridDim = dim3(static_cast<unsigned>(
      2 * (items < max_pairs ? items : static_cast<long long>(max_pairs))));
  e = cudaLaunchKernelEx(&cfg, kern, ta, tsa, tb, tsb, to != nullptr ? *to : ta,
                         args, to != nullptr ? 1 : 0, GROUP_M,
                         static_cast<int>(halves));
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int FORMAT>
cudaError_t launch_format(const CUtensorMap& ta, const CUtensorMap& tsa,
                          const CUtensorMap& tb, const CUtensorMap& tsb,
                          const CUtensorMap* to, const ProductArgs& args,
                          int max_pairs, cudaStream_t s) {
  switch (args.epilogue) {
    case OUT_BF16:
      return launch_pairs<FORMAT, OUT_BF16>(ta, tsa, tb, tsb, to, args, max_pairs, s);
    case OUT_FP32:
      return launch_pairs<FORMAT, OUT_FP32>(ta, tsa, tb, tsb, to, args, max_pairs, s);
    default:
      return launch_pairs<FORMAT, OUT_GELU_FP4>(ta, tsa, tb, tsb, nullptr, args,
                                                max_pairs, s);
  }
}

}  // namespace

cudaError_t launch_product_pairs(int format, const CUtensorMap& ta,
                                 const CUtensorMap& tsa, const CUtensorMap& tb,
                                 const CUtensorMap& tsb, const CUtensorMap* to,
                                 const ProductArgs& args, int max_pairs,
                                 cudaStream_t s) {
  return format == TPFP4_NV
             ? launch_format<TPFP4_NV>(ta, tsa, tb, tsb, to, args, max_pairs, s)
             : launch_format<TPFP4_MX>(ta, tsa, tb, tsb, to, args, max_pairs, s);
}

}  // namespace fp4
}  // namespace tpmlp
