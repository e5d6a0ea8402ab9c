// The four-bit product for few rows of A (single tokens of a few requests), and
// for products of few tiles: bound by the read of B, whose rows take the MMA's
// 128 lanes while up to 128 rows of A are its columns.
//
// A CTA takes 128 rows of B, NT rows of A and one of the cluster's ranges of K,
// so that a product of few tiles still keeps every SM loading.  Warp 0 loads
// (plain copies of whole tiles: no tensor maps to make and to fetch), warp 1 copies
// scales and issues MMAs, as in fp4_gemm.cu on one CTA; then warps 0 to 3 read
// their 32 lanes of the accumulator into shared memory, and after a cluster
// barrier the CTAs add up, row by row of A and in the CTAs' order, the partial
// sums.  One launch, no workspace, a fixed order.  Up to 8 rows of A may come as
// they are: four more warps quantise them (every CTA those of its range of K).
//
// Measured (NV, B not in L2, launches back to back): 1 x 4096 x 1024 3.5 us, 32 x
// 5120 x 20480 13.3 us (59 MB, 8.7 us at the copy rate), 32 x 20480 x 20480 42.6 us
// (236 MB, 5.5 TB/s).  Bound by the read of B and, below 100 MB, by some 4 us of
// launch, first loads, the cluster's barrier and the joint sums.
#pragma once
#include <algorithm>
#include <type_traits>

#include "fp4_gemm.cuh"
#include "fp4_load.cuh"

namespace tpmlp {
namespace fp4 {
namespace split {

using namespace gemm;

constexpr int FM = 128;            // rows of B ("features") a CTA takes
// Of A: packed, or up to 4 rows, or (bf16) up to 8.
enum Source : int { PACKED = 0, PLAIN_BF16 = 1, PLAIN_FP32 = 2, PLAIN_BF16_8 = 3 };
__host__ __device__ constexpr int threads_of(Source src) {
  return src == PACKED ? 128 : 256;
}
constexpr int MAX_SPLIT = 8;       // CTAs of a cluster

template <int FORMAT, int NT>
struct Shape {
  static constexpr uint32_t TILE = tile_bytes(FORMAT);
  static constexpr uint32_t B_BYTES = FM * 128, A_BYTES = NT * 128;
  static constexpr uint32_t STAGE = B_BYTES + A_BYTES + 2 * TILE;
  // two CTAs an SM (one with twice the stages: 32 x 5120 x 20480 18.1 us, not 13.3)
  static constexpr uint32_t BUDGET = 108 * 1024;
  static constexpr int STAGES = BUDGET / STAGE < 6 ? BUDGET / STAGE : 6;
  static constexpr int NUM_BARRIERS = 2 * STAGES + 1;
  static constexpr size_t SMEM = 1024 + size_t(STAGES) * STAGE +
                                 NUM_BARRIERS * 8 + 16;
  // tensor memory: the accumulator, then the scales of B and of A
  static constexpr uint32_t T_SB = NT;
  static constexpr uint32_t T_SA = NT + 4 * copies_per_tile(FORMAT);
  static constexpr uint32_t T_USED = T_SA + 4 * copies_per_tile(FORMAT);
  static constexpr uint32_t T_COLS = T_USED <= 128 ? 128 : 256;
  static_assert(STAGES >= 2 && SMEM <= 227 * 1024, "shared memory budget");
  static_assert(NT * FM * 4 <= STAGES * STAGE, "partial sums fit the stages");
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Four consecutive features of one row of A.
template <int FORMAT, int EPI>
__device__ __forceinline__ void finish(const ProductArgs& a, int row, int n0,
                                       int lane, float inv_gy, float (&v)[4]) {
  const int n = n0 + 4 * lane;
  const int left = a.N - n;   // features of these in the matrix
  if (a.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) v[i] += load_f32(a.bias + n + i);
  }
  if constexpr (EPI == OUT_GELU_FP4) {
    // N is a multiple of 64: a lane's four are all in the matrix or none
    gelu2_f32(v[0], v[1], a.gelu_mode);
    gelu2_f32(v[2], v[3], a.gelu_mode);
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (left <= 0) v[i] = 0.f;
      amax = max(amax, abs_bits(v[i]));
    }
    constexpr int LANES = block_size(FORMAT) / 4;   // of a block
#pragma unroll
    for (int m = 1; m < LANES; m *= 2)
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    const Scale s = block_scale<FORMAT>(amax, inv_gy);
    float q[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; i += 2)
      quotient2<FORMAT, true>(v[i], v[i + 1], s, q[i], q[i + 1]);
    uint8_t* codes = a.y.codes + code_row(row, n0 / TILE_COLS, a.y.ktiles);
    *reinterpret_cast<uint16_t*>(codes + code_unit(row, n % TILE_COLS / 32) +
                                 n % 32 / 2) = static_cast<uint16_t>(codes8(q));
    uint32_t word = s.byte << (8 * (lane / LANES % 4));
    word |= __shfl_xor_sync(0xffffffffu, word, LANES);
    word |= __shfl_xor_sync(0xffffffffu, word, 2 * LANES);
    const int kt = n / TILE_COLS;
    const int word_at = n % TILE_COLS / (4 * block_size(FORMAT));
    if (lane % (4 * LANES) == 0)
      *reinterpret_cast<uint32_t*>(
          a.y.scales + scale_word(row, kt, word_at, a.y.ktiles, tile_bytes(FORMAT))) =
          word;
    // the second half of a last k-tile that no CTA takes
    if (n0 % TILE_COLS == 0 && n0 + FM >= a.N) {
      constexpr int HALF_WORDS = 128 / (4 * block_size(FORMAT));
      reinterpret_cast<uint16_t*>(codes + code_unit(row, 4 + lane / 8))[lane % 8] =
          0;
      if (lane < HALF_WORDS)
        *reinterpret_cast<uint32_t*>(
            a.y.scales + scale_word(row, n0 / TILE_COLS, HALF_WORDS + lane,
                                    a.y.ktiles, tile_bytes(FORMAT))) =
            FORMAT == TPFP4_NV ? 0u : 0x7f7f7f7fu;
    }
    return;
  }
  if constexpr (EPI == OUT_BF16) {
    if (a.residual != nullptr) {
      const auto* r = static_cast<const __nv_bfloat16*>(a.residual) + row * a.ldr + n;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) v[i] += __bfloat162float(r[i]);
    }
    auto* out = static_cast<__nv_bfloat16*>(a.out) + row * a.ldo + n;
    if (left >= 4 && (reinterpret_cast<uintptr_t>(out) & 7u) == 0) {
      *reinterpret_cast<uint2*>(out) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) out[i] = __float2bfloat16_rn(v[i]);
    }
  } else if constexpr (EPI == OUT_FP32) {
    float* out = static_cast<float*>(a.out) + row * a.ldo + n;
    if (left >= 4 && (reinterpret_cast<uintptr_t>(out) & 15u) == 0) {
      *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) out[i] = v[i];
    }
  }
}

// Warps 4 to 7 of a product that quantises A itself, a k-tile each in turn.  A lane
// takes two (of 8 rows four) units of 16 elements, of rows lane / 16, that + 2 and so
// on, and puts their codes and scales where the copies of a packed A would; its next
// k-tile's are loaded meanwhile, so that those of eight k-tiles are in flight (with
// all warps on one k-tile, 8 x 5120 x 20480 took 16 us instead of 10).
//
// No more warps than stages: a warp's last k-tile i - QUANT_WARPS had stage
// i - QUANT_WARPS - STAGES free, so that of this stage's uses all but the last are
// over, and the parity of `empty` says whether the last is.
constexpr int QUANT_WARPS = 4;
template <int FORMAT, int NT, Source SRC>
__device__ __forceinline__ void quantize_rows(const ProductArgs& a, int k_lo,
                                              int k_hi, uint32_t s_a,
                                              uint32_t s_sa, uint32_t full0,
                                              uint32_t empty0, const Ctl& ctl) {
  using S = Shape<FORMAT, NT>;
  static_assert(QUANT_WARPS <= S::STAGES, "parities tell two phases apart");
  constexpr int UNITS = SRC == PLAIN_BF16_8 ? 4 : 2;
  using T = std::conditional_t<SRC == PLAIN_FP32, float, __nv_bfloat16>;
  const int lane = threadIdx.x & 31;
  const int unit = lane & 15, row0 = lane >> 4;
  const bool wide = (reinterpret_cast<uintptr_t>(a.x) |
                     static_cast<uintptr_t>(a.x_stride * sizeof(T))) % 16 == 0;
  const T* src = static_cast<const T*>(a.x) + row0 * a.x_stride + unit * 16;
  const float inv_g = exp2_of(-a.x_exponent);
  const Extent e = extent_of(static_cast<const T*>(a.x), a.x_stride, a.M, a.a.cols);
  auto load = [&](int i, Raw<T> (&raw)[UNITS]) {
    const int col = (k_lo + i) * TILE_COLS;
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
      if (2 * j >= a.M) break;   // both of the warp's rows
      const T* p = src + 2 * j * a.x_stride + col;
      const int n = row0 + 2 * j < a.M ? a.a.cols - col - unit * 16 : 0;
      if (wide)
        load16<T, 16>(p, n, e, raw[j]);
      else
        load16<T, 0>(p, n, e, raw[j]);
    }
  };
  auto store = [&](uint32_t stage, const Raw<T> (&raw)[UNITS]) {
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
      if (2 * j >= a.M) break;
      const int row = row0 + 2 * j;
      float v[16];
      raw[j].floats(v);
      uint32_t amax = raw[j].amax();
      if constexpr (FORMAT == TPFP4_MX)
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      const Scale s = block_scale<FORMAT>(amax, inv_g);
      const uint2 c = codes16<FORMAT, sizeof(T) == 4>(v, s);
      const uint32_t at = s_a + stage * S::A_BYTES + row * 128 +
                          code_unit(row, unit / 2) + unit % 2 * 8;
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(c.x), "r"(c.y)
                   : "memory");
      // four blocks' scale bytes in one word, as in the row kernel
      constexpr int LANES = block_size(FORMAT) / 16;   // of a block
      uint32_t word = s.byte << (8 * (lane / LANES & 3));
      word |= __shfl_xor_sync(0xffffffffu, word, LANES);
      word |= __shfl_xor_sync(0xffffffffu, word, 2 * LANES);
      if (unit % (4 * LANES) == 0)
        asm volatile(
            "st.shared.b32 [%0], %1;" ::"r"(s_sa + stage * S::TILE +
                                            unit / (4 * LANES) * 512 + row * 16),
            "r"(word)
            : "memory");
    }
  };
  Raw<T> now[UNITS], next[UNITS];
  int i = static_cast<int>(threadIdx.x >> 5) - 4;
  if (k_lo + i < k_hi) load(i, now);
  for (; k_lo + i < k_hi; i += QUANT_WARPS) {
    const uint32_t stage = static_cast<uint32_t>(i % S::STAGES);
    const uint32_t phase = static_cast<uint32_t>(i / S::STAGES) & 1u;
    if (k_lo + i + QUANT_WARPS < k_hi) load(i + QUANT_WARPS, next);
    if (!wait_warp(empty0 + 8u * stage, phase ^ 1u, ctl, ROLE_PRODUCER)) return;
    store(stage, now);
    ptx::fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(full0 + 8u * stage);
#pragma unroll
    for (int j = 0; j < UNITS; ++j) now[j] = next[j];
  }
}

template <int FORMAT, int EPI, int NT, Source SRC>
__global__ void __launch_bounds__(threads_of(SRC), 2)
    product_split_kernel(const ProductArgs args, const int split) {
  using S = Shape<FORMAT, NT>;
  constexpr int NUM_WARPS = threads_of(SRC) / 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s_b = ptx::smem_u32(smem);
  const uint32_t s_a = s_b + S::STAGES * S::B_BYTES;
  const uint32_t s_sb = s_a + S::STAGES * S::A_BYTES;
  const uint32_t s_sa = s_sb + S::STAGES * S::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + size_t(S::STAGES) * S::STAGE);
  const uint32_t full0 = ptx::smem_u32(bars);
  const uint32_t empty0 = full0 + 8u * S::STAGES;
  const uint32_t done_bar = empty0 + 8u * S::STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + S::NUM_BARRIERS);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  if (args.dependent) let_next_launch_start();
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  const int n0 = static_cast<int>(blockIdx.x) / split * FM;
  const int t0 = static_cast<int>(blockIdx.y) * NT;
  const int ktiles = args.a.ktiles;
  const int k_lo = static_cast<int>(static_cast<long long>(ktiles) * rank / split);
  const int k_hi =
      static_cast<int>(static_cast<long long>(ktiles) * (rank + 1) / split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      // the producer, and the warp that quantises A's k-tile
      ptx::mbar_init(full0 + 8u * s, SRC == PACKED ? 1 : 2);
      ptx::mbar_init(empty0 + 8u * s, 1);
    }
    ptx::mbar_init(done_bar, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), S::T_COLS);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const Ctl ctl{abort_flag, args.status, args.budget_ns};
  if (!args.dependent) {
    wait_for_launch_before();
    let_next_launch_start();
  }
  if (SRC != PACKED && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 4)
    args.a.head->status[threadIdx.x] = 0;

  // The producer alone runs ahead of the launch before: the others' bounded waits
  // start after it, so that a budget counts waits of this kernel only.
  if (SRC == PACKED && warp != 0) wait_for_launch_before();

  if (warp == 0) {
    // ------------------------------------------------------ producer --
    uint32_t stage = 0, phase = 0;
    const size_t tb0 = static_cast<size_t>(n0 / TILE_ROWS) * ktiles;
    const size_t ta0 = static_cast<size_t>(t0 / TILE_ROWS) * ktiles;
    auto load_b = [&](int kt, uint32_t st) {
      const uint32_t fb = full0 + 8u * st;
      ptx::mbar_arrive_expect_tx(
          fb, SRC == PACKED ? S::STAGE : S::B_BYTES + S::TILE);
      ptx::bulk_load_1d(s_b + st * S::B_BYTES,
                        args.b.codes + (tb0 + kt) * CODE_TILE, S::B_BYTES, fb);
      ptx::bulk_load_1d(s_sb + st * S::TILE, args.b.scales + (tb0 + kt) * S::TILE,
                        S::TILE, fb);
    };
    auto load_a = [&](int kt, uint32_t st) {
      const uint32_t fb = full0 + 8u * st;
      ptx::bulk_load_1d(s_a + st * S::A_BYTES,
                        args.a.codes + (ta0 + kt) * CODE_TILE, S::A_BYTES, fb);
      ptx::bulk_load_1d(s_sa + st * S::TILE, args.a.scales + (ta0 + kt) * S::TILE,
                        S::TILE, fb);
    };
    const int early = min(k_lo + S::STAGES, k_hi);   // B before A may be read
    if (elect_one())
      for (int kt = k_lo; kt < early; ++kt) load_b(kt, kt - k_lo);
    __syncwarp();
    if (SRC == PACKED) wait_for_launch_before();
    for (int kt = k_lo; kt < k_hi; ++kt) {
      if (!wait_warp(empty0 + 8u * stage, phase ^ 1u, ctl, ROLE_PRODUCER)) break;
      if (elect_one()) {
        if (kt >= early) load_b(kt, stage);
        if (SRC == PACKED) load_a(kt, stage);
      }
      __syncwarp();
      if (++stage == S::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------- MMA issuer --
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
    const uint64_t desc_b = ptx::sdesc_sw128(s_b, 16, 1024);
    const uint64_t desc_a = ptx::sdesc_sw128(s_a, 16, 1024);
    const uint64_t desc_sb = sdesc_scales(s_sb);
    const uint64_t desc_sa = sdesc_scales(s_sa);
    uint32_t stage = 0, phase = 0;
    for (int kt = k_lo; kt < k_hi; ++kt) {
      if (!wait_warp(full0 + 8u * stage, phase, ctl, ROLE_MMA)) break;
      ptx::tc_fence_after();
      if (elect_one()) {
        ktile_mmas<FORMAT, 1, FM, NT, 1>(
            tmem, desc_b + stage * (S::B_BYTES / 16),
            desc_a + stage * (S::A_BYTES / 16), desc_sb + stage * (S::TILE / 16),
            desc_sa + stage * (S::TILE / 16), tmem + S::T_SB, tmem + S::T_SA,
            kt == k_lo);
        ptx::mma_commit(empty0 + 8u * stage);
      }
      __syncwarp();
      if (++stage == S::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (elect_one()) ptx::mma_commit(done_bar);   // (after an abort too)
  } else if constexpr (SRC != PACKED) {
    if (warp >= 4)
      quantize_rows<FORMAT, NT, SRC>(args, k_lo, k_hi, s_a, s_sa, full0, empty0,
                                     ctl);
  }
  __syncwarp();
  // -------------------------------------------- partial sums to shared --
  // done: every MMA of this CTA has finished, and with them every copy that
  // they waited for; after an abort copies may be in flight, and the stages are
  // left alone.
  bool ok = wait_warp(done_bar, 0, ctl, ROLE_EPILOGUE);
  ok = __syncthreads_and(ok && *reinterpret_cast<volatile int*>(abort_flag) == 0);
  ptx::tc_fence_after();
  if (ok && warp < 4) {
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(warp * 32) << 16);
    float* part = reinterpret_cast<float*>(smem) + warp * 32 + lane;
    const int rows = min(NT, args.M - t0);
#pragma unroll 1
    for (int c = 0; c < NT && c < rows; c += 16) {
      uint32_t r[16];
      ptx::tmem_ld_32x32b_x16(taddr + c, r);
      ptx::tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) part[(c + i) * FM] = __uint_as_float(r[i]);
    }
  } else if (!ok && warp == 0 && lane == 0) {
    wait_teardown(done_bar, 0);
    const uint64_t t = ptx::globaltimer_ns();   // copies in flight
    while (ptx::globaltimer_ns() - t < 2000000ull) {
    }
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, S::T_COLS);
  }
  // --------------------------------------------------- sums, epilogue --
  if (SRC == PACKED) wait_for_launch_before();
  const float2 g =
      gain_factors(SRC == PACKED ? args.a.head->g : exp2_of(args.x_exponent),
                   args.b.head->g);
  float inv_gy = 1.f;
  if constexpr (EPI == OUT_GELU_FP4) {
    inv_gy = exp2_of(-args.y_exponent);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
      args.y.head->g = exp2_of(args.y_exponent);
      for (int i = 0; i < 4; ++i) args.y.head->status[i] = 0;
    }
  }
  const int rows = min(NT, args.M - t0);
  for (int t = rank * NUM_WARPS + warp; t < rows; t += NUM_WARPS * split) {
    const uint32_t at = s_b + static_cast<uint32_t>(t * FM + 4 * lane) * 4u;
    float4 p[MAX_SPLIT];
#pragma unroll
    for (int c = 0; c < MAX_SPLIT; ++c)
      if (c < split) p[c] = ld_cluster_f4(ptx::mapa_shared(at, c));
    float v[4] = {p[0].x, p[0].y, p[0].z, p[0].w};
#pragma unroll
    for (int c = 1; c < MAX_SPLIT; ++c)
      if (c < split) v[0] += p[c].x, v[1] += p[c].y, v[2] += p[c].z, v[3] += p[c].w;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = v[i] * g.x * g.y;
    finish<FORMAT, EPI>(args, t0 + t, n0, lane, inv_gy, v);
  }
  ptx::cluster_sync();   // no CTA leaves while its sums are being read
}

// (K split over clusters, not at all: 32 x 5120 x 20480 13.3 us and 25.4, 8 x 20480 x
// 5120, whose 160 CTAs fill the SMs, 13.3 and 13.1.)
// Clusters of `size` CTAs that fit at once, two CTAs to an SM, when a cluster's
// SMs come from one of eight groups of at least sms / 9.  (A rule on the SM
// count alone, so that the order of the sums, and with it the last bits, is the
// same on every GPU of a model.)
inline long long resident_clusters(int size, int sms) {
  return 8ll * (sms / 9 * 2 / size);
}

template <int FORMAT, int EPI, int NT, Source SRC>
cudaError_t launch_tokens(const ProductArgs& args, int sms, cudaStream_t s) {
  using S = Shape<FORMAT, NT>;
  auto kern = product_split_kernel<FORMAT, EPI, NT, SRC>;
  cudaError_t e = cudaFuncSetAttribute(
      kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::SMEM));
  if (e != cudaSuccess) return e;
  const long long features = (args.N + FM - 1) / FM;
  const long long tokens = (args.M + NT - 1) / NT;
  if (tokens > 65535) return cudaErrorInvalidValue;
  // as many CTAs as the SMs hold at once, and a k-tile at least for each
  int split = 1;
  for (int c = 2; c <= MAX_SPLIT && c <= args.a.ktiles; ++c)
    if (features * tokens <= resident_clusters(c, sms)) split = c;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(threads_of(SRC));
  cfg.gridDim = dim3(static_cast<unsigned>(features * split),
                     static_cast<unsigned>(tokens));
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, args, split);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace split
}  // namespace fp4
}  // namespace tpmlp
