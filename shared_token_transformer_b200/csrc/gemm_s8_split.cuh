// gemm_s8_split.cuh -- the 8-bit integer linear layer for too few output tiles.
//
// A few hundred rows give fewer 128 x 64 tiles than there are SMs, and a long K then
// runs slice by slice on a part of the machine.  Here a cluster of S CTAs (2 to 6) shares
// a tile: each takes a stretch of K into its own TMEM accumulator, and the int32 sums
// meet by distributed shared memory, where addition is exact in any order.  Each of the
// tile's four parts of sixteen accumulator columns is finished by one CTA of the
// cluster.  Bound by the slices' latency through the ring: with S stretches the chain
// is S times shorter: 257 x 4096 -> 1024 (48 tiles, S = 2) takes 8.5 us instead of 12.0,
// 128 x 4096 -> 1024 (16 tiles, S = 6) 6.3 instead of 11.7.  Only as many clusters as run
// at once are used; a second wave would cost more than splitting saves (S = 3 took 14.1 us
// on the first of these).
#pragma once

#include "gemm_s8.cuh"

namespace ts {

constexpr int kSplitMax = 6;
constexpr int kSplitBN = 64;

struct SplitSmem {
  static constexpr int STAGES = 6;
  static constexpr int A_BYTES = 128 * 128, B_BYTES = kSplitBN * 128, STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int PART = 128 * 16 * 4;                 // one part of a tile: 128 rows x 16 int32
  static constexpr int PART_OFFSET = STAGES * STAGE_BYTES;  // the other CTAs' sums of the parts this one finishes
  static constexpr int BAR_OFFSET = PART_OFFSET + (kSplitMax - 1) * PART;
  static constexpr int NBARS = 2 * STAGES + 1;
  static constexpr int BYTES = BAR_OFFSET + NBARS * 8 + 16;
  static constexpr int LAUNCH_BYTES = BYTES + 1024;
};
// CTA of a cluster of S that finishes part p, and how many parts a CTA finishes at most
__host__ __device__ constexpr int split_owner(int p, int S) { return p * S / 4; }
__host__ __device__ constexpr int split_parts(int S) { return S < 4 ? 2 : 1; }
static_assert(2 * split_parts(3) <= kSplitMax - 1 && split_parts(2) <= kSplitMax - 1, "room for the sums");

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster4(uint32_t addr, const float* v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(__float_as_uint(v[0])),
               "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3]))
               : "memory");
}
// eight consecutive columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

template <int EPI>
__global__ void __launch_bounds__(kS8Threads, 1)
    gemm_s8_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const GemmArgs args, int S) {
  using SM = SplitSmem;
  constexpr int STAGES = SM::STAGES, BN = kSplitBN, KE = 128;
  constexpr bool GLU = EPI == EPI_SWIGLU;
  constexpr uint32_t IDESC = idesc_make(1u, BN, 128, 2u);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_full = sbase + SM::BAR_OFFSET;
  const uint32_t bar_empty = bar_full + 8 * STAGES;
  const uint32_t bar_tfull = bar_empty + 8 * STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::BAR_OFFSET + SM::NBARS * 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), tile = static_cast<int>(blockIdx.x) / S;
  const int mt = (args.M + 127) / 128, m0 = tile % mt * 128, n0 = tile / mt * BN;
  const int KB = (args.K + KE - 1) / KE;
  const int kb0 = static_cast<int>(static_cast<long long>(KB) * rank / S);          // this CTA's slices (S <= KB)
  const int kb1 = static_cast<int>(static_cast<long long>(KB) * (rank + 1) / S);

  if (warp == kS8TmaWarp && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    mbar_init(bar_tfull, 1);
    fence_barrier_init();
  }
  if (warp == kS8MmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();         // waited for below, before the first access to another CTA's shared memory
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  // epilogue warps: lane quarter warp % 4 (one row per lane), part warp / 4: sixteen accumulator columns (SwiGLU: eight
  // gate columns and their eight up columns)
  const int quarter = warp & 3, part = warp >> 2;
  const int row = m0 + quarter * 32 + lane;
  const int n_out = GLU ? args.N / 2 : args.N;
  const int col = GLU ? n0 / 2 + part * 8 : n0 + part * 16;
  const bool epi = warp < kS8EpiWarps;
  const int owner = split_owner(part, S);
  const bool mine = epi && owner == rank;
  float acc[16], ws[16], bi[16], rs = 0.f;
  if (warp == kS8TmaWarp) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const uint32_t s = it % STAGES;
        if (it >= STAGES && !mbar_wait(bar_empty + 8 * s, ((it / STAGES) - 1) & 1)) { ok = false; break; }
        const uint32_t sa = sbase + s * SM::STAGE_BYTES;
        mbar_expect_tx(bar_full + 8 * s, SM::STAGE_BYTES);
        tma_load_2d(sa, &tmA, bar_full + 8 * s, kb * KE, m0);
        if (GLU) {
          tma_load_2d(sa + SM::A_BYTES, &tmB, bar_full + 8 * s, kb * KE, n0 / 2);
          tma_load_2d(sa + SM::A_BYTES + SM::B_BYTES / 2, &tmB, bar_full + 8 * s, kb * KE, args.N / 2 + n0 / 2);
        } else {
          tma_load_2d(sa + SM::A_BYTES, &tmB, bar_full + 8 * s, kb * KE, n0);
        }
      }
      // no copy may still be landing when the CTA exits (matters only after a timeout)
      for (uint32_t n = ok ? it : it > STAGES ? it - STAGES : 0; n < it; ++n) mbar_wait(bar_full + 8 * (n % STAGES), (n / STAGES) & 1);
    }
    __syncwarp();
  } else if (warp == kS8MmaWarp) {
    if (lane == 0) {
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        const uint32_t it = kb - kb0, s = it % STAGES;
        if (!mbar_wait(bar_full + 8 * s, (it / STAGES) & 1)) { ok = false; break; }
        tc_fence_after();
        const uint32_t sa = sbase + s * SM::STAGE_BYTES;
        const uint64_t da = sdesc_sw128(sa), db = sdesc_sw128(sa + SM::A_BYTES);
#pragma unroll
        for (int k = 0; k < KE / 32; ++k) tc_mma_i8(tmem, da + 2 * k, db + 2 * k, IDESC, (it | k) != 0);
        tc_commit(bar_empty + 8 * s);
      }
      if (ok) tc_commit(bar_tfull);
    }
    __syncwarp();
  } else {
    // what the outputs need arrives while the accumulator fills
    if (mine) {
      if (row < args.M) rs = __ldg(args.a_scale + row);
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        // SwiGLU: values 0-7 belong to the gate columns, 8-15 to the up columns
        const int c = GLU ? (i < 8 ? 0 : n_out) + min(col + (i & 7), n_out - 4) : min(col + i, n_out - 4);
        const float4 w4 = __ldg(reinterpret_cast<const float4*>(args.w_scale + c));
        const float4 b4 = __ldg(reinterpret_cast<const float4*>(args.bias + c));
        ws[i] = w4.x; ws[i + 1] = w4.y; ws[i + 2] = w4.z; ws[i + 3] = w4.w;
        bi[i] = b4.x; bi[i + 1] = b4.y; bi[i + 2] = b4.z; bi[i + 3] = b4.w;
      }
    }
    __all_sync(0xffffffffu, mbar_wait(bar_tfull, 0));    // after a timeout (reported) the sums are worthless but safe
    tc_fence_after();
    const uint32_t trow = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    if (GLU) {
      tmem_ld8(trow + part * 8, acc);
      tmem_ld8(trow + BN / 2 + part * 8, acc + 8);
    } else {
      tmem_ld16(trow + part * 16, acc);
    }
    tmem_wait_ld();
  }
  cluster_wait();           // every CTA of the cluster runs
  // slot of a source CTA in the owner's room, and of a part among those the owner finishes; sums lie as four 16-byte
  // quads of a row, each quad's rows side by side
  auto sums = [&](int src) -> uint32_t {
    const int slot = src < owner ? src : src - 1;
    int first = part;
    while (first > 0 && split_owner(first - 1, S) == owner) --first;
    return sbase + SM::PART_OFFSET + (slot * split_parts(S) + part - first) * SM::PART + (quarter * 32 + lane) * 16;
  };
  if (epi && !mine) {
    const uint32_t dst = cluster_map(sums(rank), static_cast<uint32_t>(owner));
#pragma unroll
    for (int q = 0; q < 4; ++q) st_cluster4(dst + q * 2048, acc + 4 * q);
  }
  cluster_arrive();
  cluster_wait();           // the sums have arrived; no CTA touches another's shared memory from here on
  if (mine) {
    for (int src = 0; src < S; ++src) {
      if (src == rank) continue;
      const uint8_t* p = smem + (sums(src) - sbase);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int4 v = *reinterpret_cast<const int4*>(p + q * 2048);
        acc[4 * q] = __int_as_float(__float_as_int(acc[4 * q]) + v.x);
        acc[4 * q + 1] = __int_as_float(__float_as_int(acc[4 * q + 1]) + v.y);
        acc[4 * q + 2] = __int_as_float(__float_as_int(acc[4 * q + 2]) + v.z);
        acc[4 * q + 3] = __int_as_float(__float_as_int(acc[4 * q + 3]) + v.w);
      }
    }
    s8_dequant<16>(acc, ws, bi, rs);
    constexpr int OUT = GLU ? 8 : 16;
    if (EPI == EPI_GELU || GLU) {
#pragma unroll
      for (int i = 0; i < OUT; i += 2) {
        const uint64_t z = pack_f32x2(acc[i], acc[i + 1]);
        const uint64_t y = GLU ? silu_mul2(z, pack_f32x2(acc[8 + i & 15], acc[9 + i & 15])) : gelu_exp2(z);
        acc[i] = lo_f32(y);
        acc[i + 1] = hi_f32(y);
      }
    }
    if (row < args.M) {
      bf16* y = args.out + static_cast<size_t>(row) * args.ldo + col;
#pragma unroll
      for (int i = 0; i < OUT; i += 8) {
        if (col + i >= n_out) break;
        if (EPI == EPI_RESID) {
          float r[8];
          bf16x8_to_f32(*reinterpret_cast<const uint4*>(y + i), r);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[i + e] += r[e];
        }
        *reinterpret_cast<uint4*>(y + i) = f32_to_bf16x8(acc + i);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kS8MmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, BN);
  }
}

}  // namespace ts
