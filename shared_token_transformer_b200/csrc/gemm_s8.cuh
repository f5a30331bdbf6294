// gemm_s8.cuh -- linear layers with signed 8-bit integer operands.
//
//   Y[m, n] = epi( (sum_k A[m, k] W[n, k]) * a_scale[m] * w_scale[n] + b[n] )
//
// A [M, K] and W [N, K] hold signed bytes, the sums are exact in int32 (tcgen05
// kind::i8, 32 products along K per instruction), and the epilogues are those of the
// bf16 and e4m3 GEMMs (gemm_tc.cuh).  Any K % 16 == 0 and N % 8 == 0: the copies fill
// K past the end with zeros and clip columns past N.
//
// The pipeline is gemm_tc.cuh's: a persistent grid walks the output tiles, one warp
// feeds 128-byte K slices by TMA into a ring, one lane issues the MMAs into one of two
// TMEM accumulators while the epilogue warps drain the other.  An integer tile takes
// half as long as a bf16 tile of the same K, so the epilogue decides:
//   - sixteen epilogue warps, four per scheduler, each with boxes of 32 rows and 32
//     columns that it stages and stores on its own, without a barrier between warps
//     (2 KB each, so that five ring stages fit: with four, the K = 6144 product took
//     107 us instead of 91 at 14086 x 1536);
//   - the arithmetic in packed f32x2;
//   - the columns' scales and biases come by bulk copy into shared memory, a tile ahead
//     (read from global memory they missed L1, which the ring leaves little of).
#pragma once

#include "gemm_tc.cuh"

namespace ts {

constexpr int kS8EpiWarps = 16;
constexpr int kS8TmaWarp = kS8EpiWarps;
constexpr int kS8MmaWarp = kS8EpiWarps + 1;
constexpr int kS8Threads = 32 * (kS8EpiWarps + 2);

// Output columns of an epilogue warp's box: 32, or one head for QKV.
template <int EPI>
constexpr int s8_box() {
  return EPI == EPI_QKV ? 64 : 32;
}

template <int BN, int STAGES, int EPI, int CG>
struct S8Smem {
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = (BN / CG) * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int BOX_BYTES = 32 * s8_box<EPI>() * 2;
  static constexpr int EPI_OFFSET = STAGES * STAGE_BYTES;                    // one box per epilogue warp
  static constexpr int VEC_OFFSET = EPI_OFFSET + kS8EpiWarps * BOX_BYTES;    // 2 x (scales [BN], biases [BN])
  static constexpr int VEC_BYTES = 2 * BN * 4;
  static constexpr int BAR_OFFSET = VEC_OFFSET + 2 * VEC_BYTES;
  // full, empty; accumulators full, empty; vectors full, empty (two each); residual boxes
  static constexpr int NBARS = 2 * STAGES + 8 + kS8EpiWarps;
  static constexpr int BYTES = BAR_OFFSET + NBARS * 8 + 16;
  static constexpr int LAUNCH_BYTES = BYTES + 1024;
  static_assert(LAUNCH_BYTES <= 227 * 1024, "shared memory of one CTA");
};

// W columns of a row: v (int32 accumulators as TMEM returned them) becomes acc * (rs * w_scale) + bias.  ws and b
// are the columns' vectors in shared memory.
template <int W>
__device__ __forceinline__ void s8_dequant(float* v, const float* ws, const float* b, float rs) {
  const uint64_t rs2 = splat_f32x2(rs);
#pragma unroll
  for (int i = 0; i < W; i += 4) {
    const float4 w4 = *reinterpret_cast<const float4*>(ws + i);
    const float4 b4 = *reinterpret_cast<const float4*>(b + i);
    const uint64_t a0 = pack_f32x2(__int2float_rn(__float_as_int(v[i])), __int2float_rn(__float_as_int(v[i + 1])));
    const uint64_t a1 = pack_f32x2(__int2float_rn(__float_as_int(v[i + 2])), __int2float_rn(__float_as_int(v[i + 3])));
    const uint64_t z0 = fma_f32x2(a0, mul_f32x2(pack_f32x2(w4.x, w4.y), rs2), pack_f32x2(b4.x, b4.y));
    const uint64_t z1 = fma_f32x2(a1, mul_f32x2(pack_f32x2(w4.z, w4.w), rs2), pack_f32x2(b4.z, b4.w));
    v[i] = lo_f32(z0);
    v[i + 1] = hi_f32(z0);
    v[i + 2] = lo_f32(z1);
    v[i + 3] = hi_f32(z1);
  }
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {   // the larger, NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// GELU of a pair:
//   x (1 + erf(x / sqrt 2)) / 2 = max(x, 0) - a 2^Q(a),   a = |x|,   2^Q(a) = erfc(a / sqrt 2) / 2
// with Q a polynomial of degree 6 fitted here over [0, 8] (Lawson's iteration, each error weighted by what it does to
// the GELU): within 1.4e-7 of exact-erf GELU relative to max(1, |GELU|), in fp32 arithmetic.  a ends at 8, where the
// second term is 5e-15.  Seven multiply-adds and one exponential per value; -a serves as the argument, so that no sign
// has to be put back.
__device__ __forceinline__ uint64_t gelu_exp2(uint64_t x2) {
  const float x0 = lo_f32(x2), x1 = hi_f32(x2);
  const uint64_t na = pack_f32x2(fmaxf(-fabsf(x0), -8.f), fmaxf(-fabsf(x1), -8.f));
  const uint64_t relu = pack_f32x2(max_nan(x0, 0.f), max_nan(x1, 0.f));    // carries a NaN into the result
  uint64_t q = fma_f32x2(splat_f32x2(2.9704213375225663e-05f), na, splat_f32x2(0.0007424539653584361f));
  q = fma_f32x2(q, na, splat_f32x2(0.008002202026546001f));
  q = fma_f32x2(q, na, splat_f32x2(0.05330503359436989f));
  q = fma_f32x2(q, na, splat_f32x2(-0.45884037017822266f));
  q = fma_f32x2(q, na, splat_f32x2(1.1511822938919067f));
  q = fma_f32x2(q, na, splat_f32x2(5.265353138383944e-06f - 1.0f));
  return fma_f32x2(na, pack_f32x2(ex2_approx(lo_f32(q)), ex2_approx(hi_f32(q))), relu);
}
// silu(g) * u of a pair: g / (1 + 2^(-g log2 e)) by the approximate exponential and reciprocal; the limit of a
// large negative g, whose 2^x is infinite, is -0
__device__ __forceinline__ uint64_t silu_mul2(uint64_t g, uint64_t u) {
  const uint64_t x = mul_f32x2(g, splat_f32x2(-1.4426950408889634f));
  const uint64_t den = add_f32x2(pack_f32x2(ex2_approx(lo_f32(x)), ex2_approx(hi_f32(x))), splat_f32x2(1.0f));
  return mul_f32x2(mul_f32x2(g, pack_f32x2(rcp_approx(lo_f32(den)), rcp_approx(hi_f32(den)))), u);
}

template <int BN, int STAGES, int EPI, int R0, int R1, int R2, int CG>
__global__ void __launch_bounds__(kS8Threads, 1)
    gemm_s8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmD, const GemmArgs args) {
  using SM = S8Smem<BN, STAGES, EPI, CG>;
  constexpr uint32_t TMEM_COLS = 2 * BN;
  constexpr uint32_t IDESC = idesc_make(1u, BN, 128 * CG, 2u);
  constexpr int TM = 128 * CG;
  constexpr int KE = 128;
  constexpr bool GLU = EPI == EPI_SWIGLU;
  constexpr int BO = GLU ? BN / 2 : BN;           // output columns per tile
  constexpr int CW = s8_box<EPI>();               // output columns of a warp's box
  constexpr int NB = BO > 4 * CW ? BO / (4 * CW) : 1;   // boxes of a warp per tile, side by side
  static_assert(!GLU || BN >= 128, "SwiGLU tiles hold at least 64 outputs");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_full = sbase + SM::BAR_OFFSET;
  const uint32_t bar_empty = bar_full + 8 * STAGES;
  const uint32_t bar_tfull = bar_empty + 8 * STAGES;
  const uint32_t bar_tempty = bar_tfull + 16;
  const uint32_t bar_vfull = bar_tempty + 16;
  const uint32_t bar_vempty = bar_vfull + 16;
  const uint32_t bar_resid = bar_vempty + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::BAR_OFFSET + SM::NBARS * 8);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int mt = (args.M + TM - 1) / TM;
  const int nt = (args.N + BN - 1) / BN;
  const int ntiles = mt * nt;
  const int KB = (args.K + KE - 1) / KE;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int unit = CG == 2 ? static_cast<int>(blockIdx.x) / 2 : static_cast<int>(blockIdx.x);
  const int units = CG == 2 ? static_cast<int>(gridDim.x) / 2 : static_cast<int>(gridDim.x);
  const bool leader = rank == 0;

  if (warp == kS8TmaWarp && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmD);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_tfull + 8 * b, 1);
      mbar_init(bar_tempty + 8 * b, kS8EpiWarps * CG);
      mbar_init(bar_vfull + 8 * b, 1);
      mbar_init(bar_vempty + 8 * b, kS8EpiWarps);
    }
    for (int w = 0; w < kS8EpiWarps; ++w) mbar_init(bar_resid + 8 * w, 1);
    fence_barrier_init();
  }
  if (warp == kS8MmaWarp) {
    if (CG == 2) {
      tmem_alloc2(smem_u32(tmem_slot), TMEM_COLS);
      tmem_relinquish2();
    } else {
      tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  if (warp == kS8TmaWarp) {
    if (lane == 0) {
      uint32_t it = 0, j = 0;
      bool ok = true;
      for (int tile = unit; tile < ntiles && ok; tile += units, ++j) {
        int m0, n0;
        gemm_tile_origin(tile, mt, nt, BN, m0, n0, TM);
        for (int kb = 0; kb < KB; ++kb, ++it) {
          const uint32_t s = it % STAGES;
          if (it >= STAGES && !mbar_wait(bar_empty + 8 * s, ((it / STAGES) - 1) & 1)) { ok = false; break; }
          const uint32_t sa = sbase + s * SM::STAGE_BYTES;
          if (CG == 2) {
            const uint32_t fb = cluster_map(bar_full + 8 * s, 0);
            if (leader) mbar_expect_tx(bar_full + 8 * s, 2 * SM::STAGE_BYTES);
            tma_load_2d_pair(sa, &tmA, fb, kb * KE, m0 + static_cast<int>(rank) * 128);
            if (GLU)    // the even CTA holds the BN/2 gate rows, the odd one the BN/2 up rows
              tma_load_2d_pair(sa + SM::A_BYTES, &tmB, fb, kb * KE, (rank ? args.N / 2 : 0) + n0 / 2);
            else
              tma_load_2d_pair(sa + SM::A_BYTES, &tmB, fb, kb * KE, n0 + static_cast<int>(rank) * (BN / 2));
          } else {
            mbar_expect_tx(bar_full + 8 * s, SM::STAGE_BYTES);
            tma_load_2d(sa, &tmA, bar_full + 8 * s, kb * KE, m0);
            if (GLU) {
              tma_load_2d(sa + SM::A_BYTES, &tmB, bar_full + 8 * s, kb * KE, n0 / 2);
              tma_load_2d(sa + SM::A_BYTES + (BN / 2) * 128, &tmB, bar_full + 8 * s, kb * KE, args.N / 2 + n0 / 2);
            } else {
              tma_load_2d(sa + SM::A_BYTES, &tmB, bar_full + 8 * s, kb * KE, n0);
            }
          }
        }
        // the tile's scales and biases (SwiGLU: those of the gate columns, then of the up columns), behind its
        // operands: the epilogue of the tile before last has to be done with the buffer
        if (!ok) break;
        const uint32_t vb = j & 1, vbar = bar_vfull + 8 * vb;
        if (j >= 2 && !mbar_wait(bar_vempty + 8 * vb, ((j >> 1) - 1) & 1)) { ok = false; break; }
        const uint32_t dst = sbase + SM::VEC_OFFSET + vb * SM::VEC_BYTES;
        const int c0 = GLU ? n0 / 2 : n0, n_out = GLU ? args.N / 2 : args.N;
        const uint32_t bytes = 4u * static_cast<uint32_t>(min(BO, n_out - c0));
        mbar_expect_tx(vbar, (GLU ? 4 : 2) * bytes);
        bulk_load(dst, args.w_scale + c0, bytes, vbar);
        bulk_load(dst + 4 * BN, args.bias + c0, bytes, vbar);
        if (GLU) {
          bulk_load(dst + 2 * BN, args.w_scale + n_out + c0, bytes, vbar);
          bulk_load(dst + 6 * BN, args.bias + n_out + c0, bytes, vbar);
        }
      }
      // no copy may still be landing when the CTA exits (matters only after a timeout; of a pair the even CTA waits for
      // both, and the odd one leaves after it)
      if (!ok) {
        if (leader)
          for (uint32_t n = it > STAGES ? it - STAGES : 0; n < it; ++n) mbar_wait(bar_full + 8 * (n % STAGES), (n / STAGES) & 1);
        for (uint32_t n = j > 2 ? j - 2 : 0; n < j; ++n) mbar_wait(bar_vfull + 8 * (n & 1), (n >> 1) & 1);
      }
    }
  } else if (warp == kS8MmaWarp) {
    if (lane == 0 && leader) {
      uint32_t it = 0, j = 0;
      bool ok = true;
      for (int tile = unit; tile < ntiles && ok; tile += units, ++j) {
        const uint32_t acc = j & 1, use = j >> 1;
        if (j >= 2 && !mbar_wait(bar_tempty + 8 * acc, (use - 1) & 1)) { ok = false; break; }
        tc_fence_after();
        const uint32_t dt = tmem + acc * BN;
        for (int kb = 0; kb < KB; ++kb, ++it) {
          const uint32_t s = it % STAGES;
          if (!mbar_wait(bar_full + 8 * s, (it / STAGES) & 1)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = sbase + s * SM::STAGE_BYTES;
          const uint64_t da = sdesc_sw128(sa);
          const uint64_t db = sdesc_sw128(sa + SM::A_BYTES);
#pragma unroll
          for (int k = 0; k < KE / 32; ++k) {
            if (CG == 2)
              tc_mma_i8_pair(dt, da + 2 * k, db + 2 * k, IDESC, (kb | k) != 0);
            else
              tc_mma_i8(dt, da + 2 * k, db + 2 * k, IDESC, (kb | k) != 0);
          }
          if (CG == 2)
            tc_commit_pair(bar_empty + 8 * s);
          else
            tc_commit(bar_empty + 8 * s);
        }
        if (!ok) break;
        if (CG == 2)
          tc_commit_pair(bar_tfull + 8 * acc);
        else
          tc_commit(bar_tfull + 8 * acc);
      }
    }
  } else {
    // epilogue warps: lane quarter warp % 4 (one row per lane), columns (warp / 4) * NB * CW .. of the tile's outputs
    const int quarter = warp & 3;
    const int bc = (warp >> 2) * (NB * CW);
    const uint32_t rbar = bar_resid + 8 * warp;
    const uint32_t stg = sbase + SM::EPI_OFFSET + warp * SM::BOX_BYTES;
    // staged rows of 2 CW bytes, swizzled as the output map reads them: 16-byte piece q of row r sits at piece
    // q ^ (r % 8) (128-byte rows) or q ^ (r / 2 % 4) (64-byte rows)
    uint8_t* srow = smem + SM::EPI_OFFSET + warp * SM::BOX_BYTES + lane * (CW * 2);
    const int sx = CW == 64 ? (lane & 7) : ((lane >> 1) & 3);
    auto piece = [&](int q) { return reinterpret_cast<uint4*>(srow + ((q ^ sx) << 4)); };
    uint32_t nload = 0, nres = 0, j = 0;   // residual boxes asked for and waited for
    const int n_out = GLU ? args.N / 2 : args.N;
    const uint32_t tempty = CG == 2 ? cluster_map(bar_tempty, 0) : bar_tempty;
    auto release = [&](uint32_t acc) {      // this warp's last TMEM read of the tile is done
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2)
          mbar_arrive_cluster(tempty + 8 * acc);
        else
          mbar_arrive(tempty + 8 * acc);
      }
    };
    for (int tile = unit; tile < ntiles; tile += units, ++j) {
      const uint32_t acc = j & 1, use = j >> 1;
      int m0, n0;
      gemm_tile_origin(tile, mt, nt, BN, m0, n0, TM);
      m0 += static_cast<int>(rank) * 128;
      const int row0 = m0 + quarter * 32, row = row0 + lane;
      const int col = (GLU ? n0 / 2 : n0) + bc;   // first output column of the warp
      const bool mine = bc < BO && row0 < args.M && col < n_out;
      // what the row needs arrives while the accumulator fills
      float rs = 1.f;
      if (row < args.M) rs = __ldg(args.a_scale + row);
      int4 pos = make_int4(0, 0, 0, 0);
      if (EPI == EPI_QKV && row < args.M) pos = __ldg(args.pos + row);
      auto load_residual = [&](int c) {
        if (lane == 0) {
          bulk_wait_read_all();                   // the last store has been read out of the staging buffer
          mbar_expect_tx(rbar, SM::BOX_BYTES);
          tma_load_2d(stg, &tmD, rbar, c, row0);
        }
        ++nload;
      };
      if (EPI == EPI_RESID && mine) load_residual(col);
      bool ok = mbar_wait(bar_vfull + 8 * acc, use & 1) && mbar_wait(bar_tfull + 8 * acc, use & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const float* ws = reinterpret_cast<const float*>(smem + SM::VEC_OFFSET + acc * SM::VEC_BYTES) + bc;
      const float* bi = ws + BN;
      const uint32_t tcol = tmem + acc * BN + (static_cast<uint32_t>(quarter * 32) << 16) + bc;
      if (!mine) release(acc);
      if (mine) {
        uint32_t pk[CW / 2];
        // out with the packed box through the staging buffer
        auto store_box = [&](int c) {
          if (EPI != EPI_RESID) {                 // the last store has been read out
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
          }
#pragma unroll
          for (int q = 0; q < CW / 8; ++q) *piece(q) = make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmD, stg, c, row0);     // rows past M and columns past N are clipped by the copy
            bulk_commit();
          }
        };
        if (EPI == EPI_QKV) {
          float v[64];
          tmem_ld32(tcol, v);
          tmem_ld32(tcol + 32, v + 32);
          tmem_wait_ld();
          release(acc);
          s8_dequant<64>(v, ws, bi, rs);
          if (col < 2 * args.d)
            qk_norm_rope64<R0, R1, R2>(v, col < args.d ? args.q_g : args.k_g, args.eps_qk, pos, args);
#pragma unroll
          for (int i = 0; i < CW; i += 2) pk[i / 2] = pack_bf16(v[i], v[i + 1]);
          store_box(col);
        } else if (GLU) {
#pragma unroll
          for (int h = 0; h < CW; h += 16) {
            float g[16], u[16];
            tmem_ld16(tcol + h, g);
            tmem_ld16(tcol + BN / 2 + h, u);
            tmem_wait_ld();
            if (h + 16 == CW) release(acc);
            s8_dequant<16>(g, ws + h, bi + h, rs);
            s8_dequant<16>(u, ws + BN / 2 + h, bi + BN / 2 + h, rs);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const uint64_t y = silu_mul2(pack_f32x2(g[i], g[i + 1]), pack_f32x2(u[i], u[i + 1]));
              pk[(h + i) / 2] = pack_bf16(lo_f32(y), hi_f32(y));
            }
          }
          store_box(col);
        } else {
          // sixteen columns at a time, the next sixteen on their way
          float v[2][16];
          tmem_ld16(tcol, v[0]);
#pragma unroll
          for (int h = 0; h < NB * CW; h += 16) {
            float* w = v[(h >> 4) & 1];
            tmem_wait_ld();
            if (h + 16 < NB * CW)
              tmem_ld16(tcol + h + 16, v[((h >> 4) + 1) & 1]);
            else
              release(acc);
            s8_dequant<16>(w, ws + h, bi + h, rs);
            if (EPI == EPI_GELU) {
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                const uint64_t y = gelu_exp2(pack_f32x2(w[i], w[i + 1]));
                w[i] = lo_f32(y);
                w[i + 1] = hi_f32(y);
              }
            } else if (EPI == EPI_RESID) {
              if (h % CW == 0) {
                ok = mbar_wait(rbar, nres & 1) && ok;
                ++nres;
              }
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                float r[8];
                bf16x8_to_f32(*piece(h % CW / 8 + q), r);
#pragma unroll
                for (int e = 0; e < 8; ++e) w[8 * q + e] += r[e];
              }
            }
#pragma unroll
            for (int i = 0; i < 16; i += 2) pk[(h % CW + i) / 2] = pack_bf16(w[i], w[i + 1]);
            if ((h + 16) % CW == 0) {
              const int c = col + h + 16 - CW;    // the box's first column
              if (c < n_out) store_box(c);
              if (EPI == EPI_RESID && h + 16 < NB * CW) {
                __syncwarp();
                load_residual(c + CW);            // zeros past N
              }
            }
          }
        }
      }
      if (EPI == EPI_RESID && !__all_sync(0xffffffffu, ok)) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_vempty + 8 * acc);
    }
    if (lane == 0) {
      if (EPI == EPI_RESID && nload != nres) mbar_wait(rbar, nres & 1);   // after a timeout: the load in flight
      bulk_wait_all();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();      // neither CTA leaves while the pair's MMAs or arrivals may still touch it
  if (warp == kS8MmaWarp) {
    tc_fence_after();
    if (CG == 2)
      tmem_dealloc2(tmem, TMEM_COLS);
    else
      tmem_dealloc(tmem, TMEM_COLS);
  }
}

}  // namespace ts
