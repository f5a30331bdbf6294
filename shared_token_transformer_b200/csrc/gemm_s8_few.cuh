// gemm_s8_few.cuh -- the 8-bit integer linear layer for few rows.
//
//   y[m, n] = epi( (sum_k x[m, k] W[n, k]) * x_scale[m] * w_scale[n] + b[n] ),  M <= 8 NT
//
// With few rows the layer is one pass over W: bound by how many bytes of W are on their
// way, not by the tensor cores.  So there is no staging: a block takes sixteen output
// columns (sixteen rows of W, and the sixteen up rows for SwiGLU), its warps split K,
// and each lane loads 32 bytes of a row of W and of a token (four lanes a 128-byte
// line) straight into the registers of the warp-wide 16 x 8 x 32 product of signed
// bytes.  The sum over k may be taken in any order as long as both operands agree, so
// the eight words of a lane's 32 bytes serve as the fragments of four products as they
// come.  The warps' int32 sums meet in shared memory.
//
// With QUANT the rows arrive as bf16 (M <= 8, and K within one round of the block's
// chunks) and every block quantises them itself (row_quant_s8) in the registers that its
// products read: the rows are few and in L2, and the call is one launch.
#pragma once

#include "gemm_s8.cuh"
#include "rowops.cuh"

namespace ts {

struct GemmFewArgs {
  int M, N, K;             // N: output columns
  const uint8_t* W;        // [N, K] ([2N, K] for SwiGLU)
  const uint8_t* x;        // [M, K] signed bytes
  const bf16* xf;          // QUANT: [M, K] bf16
  const float* x_scale;    // [M] (not with QUANT)
  const float* w_scale;    // [N] ([2N])
  const float* bias;       // [N] ([2N])
  bf16* out;               // [M, N]; the residual for EPI_RESID
  int wide;                // K % 32 == 0, W and x 32-byte aligned
  int early;               // W may be read before the previous kernel of the stream has finished (not with QUANT)
};

// The 32 bytes at p, of which `left` (a multiple of 16, or less than 1) belong to the row; zeros behind them.  wide: p
// is 32-byte aligned.
struct Bytes32 {
  uint32_t w[8];
};
template <bool STREAM>     // STREAM: read once, past L1
__device__ __forceinline__ Bytes32 load32(const uint8_t* p, int left, bool wide) {
  Bytes32 v;
  if (wide && left >= 32) {
    if (STREAM)
      asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                     "=r"(v.w[7])
                   : "l"(p));
    else
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                     "=r"(v.w[7])
                   : "l"(p));
    return v;
  }
  const uint4 z = make_uint4(0, 0, 0, 0);
  const uint4 a = left >= 16 ? *reinterpret_cast<const uint4*>(p) : z;
  const uint4 b = left >= 32 ? *reinterpret_cast<const uint4*>(p + 16) : z;
  v.w[0] = a.x; v.w[1] = a.y; v.w[2] = a.z; v.w[3] = a.w;
  v.w[4] = b.x; v.w[5] = b.y; v.w[6] = b.z; v.w[7] = b.w;
  return v;
}
// c += A (16 x 32 signed bytes) * B (32 x 8): rows of A are columns of the output, columns of B are tokens
__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 32 bf16 values of a row at p, of which `left` (a multiple of 16, or less than 1) belong to it; zeros behind them
struct Bf32 {
  uint4 v[4];
};
__device__ __forceinline__ Bf32 load_bf32(const bf16* p, int left) {
  Bf32 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.v[i] = left >= 16 * (i / 2 + 1) ? __ldg(reinterpret_cast<const uint4*>(p) + i) : make_uint4(0, 0, 0, 0);
  return r;
}

template <int NT, int EPI, bool QUANT, int WARPS, int U>
__global__ void __launch_bounds__(32 * WARPS) gemm_s8_few_kernel(const GemmFewArgs a) {
  constexpr bool GLU = EPI == EPI_SWIGLU;
  constexpr int MG = GLU ? 2 : 1;
  static_assert(!QUANT || NT == 1, "a block quantises at most eight rows");
  __shared__ int red[WARPS][MG][NT][4][32];
  __shared__ uint32_t tops[QUANT ? WARPS : 1][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, kq = (lane & 3) * 32;
  const int n0 = blockIdx.x * 16;
  // rows g and g + 8 of each group of sixteen; past N the last row again, whose outputs are not stored
  const uint8_t* wrow[MG][2];
#pragma unroll
  for (int i = 0; i < MG; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      wrow[i][h] = a.W + (static_cast<size_t>(i) * a.N + min(n0 + g + 8 * h, a.N - 1)) * a.K + kq;
  if (!a.early) pdl_wait();
  // a warp takes U chunks of 128 bytes side by side, the warps take turns
  Bytes32 wv[U][MG][2];
  auto load_w = [&](int k0) {
#pragma unroll
    for (int i = 0; i < MG; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int u = 0; u < U; ++u) wv[u][i][h] = load32<true>(wrow[i][h] + k0 + u * 128, a.K - (k0 + u * 128 + kq), a.wide);
  };
  int k0 = warp * U * 128;
  load_w(k0);
  // what this thread's outputs need: element e of the block is column e % 16 of token e / 16
  constexpr int NE = (NT * 128 + 32 * WARPS - 1) / (32 * WARPS);
  float ws[NE][MG], bi[NE][MG], xs[NE];
#pragma unroll
  for (int q = 0; q < NE; ++q) {
    const int n = min(n0 + (static_cast<int>(threadIdx.x) & 15), a.N - 1);
#pragma unroll
    for (int i = 0; i < MG; ++i) {
      ws[q][i] = __ldg(a.w_scale + i * a.N + n);
      bi[q][i] = __ldg(a.bias + i * a.N + n);
    }
  }
  if (a.early) pdl_wait();
  pdl_trigger();
  constexpr int ROUND = WARPS * U * 128;   // bytes of K that the block's chunks cover at a time
  int acc[MG][NT][4] = {};
  Bf32 xb[QUANT ? U : 1];
  RowQuantS8 rq{};
  const bf16* xf = QUANT ? a.xf + static_cast<size_t>(min(g, a.M - 1)) * a.K + kq : nullptr;
  if (QUANT) {
    // largest magnitude of row g: over this lane's chunks, the four lanes of a row, the warps
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) xb[u] = load_bf32(xf + k0 + u * 128, a.K - (k0 + u * 128 + kq));
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, bf16x8_abs_bits(xb[u].v[i]));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if ((lane & 3) == 0) tops[warp][g] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) top = max(top, tops[w][g]);
    rq = row_quant_s8(top);
    const int m = threadIdx.x >> 4;        // the row of this thread's output
    uint32_t mine = 0;
    if (m < 8) {
#pragma unroll
      for (int w = 0; w < WARPS; ++w) mine = max(mine, tops[w][m]);
    }
#pragma unroll
    for (int q = 0; q < NE; ++q) xs[q] = row_quant_s8(mine).scale;
  } else {
#pragma unroll
    for (int q = 0; q < NE; ++q) xs[q] = a.x_scale[min((static_cast<int>(threadIdx.x) + q * 32 * WARPS) >> 4, a.M - 1)];
  }
  for (; k0 < a.K; k0 += ROUND) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint8_t* xr = a.x + static_cast<size_t>(min(nt * 8 + g, a.M - 1)) * a.K + kq;
      Bytes32 xv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (QUANT) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint2 q = bf16x8_to_s8(xb[u].v[i], rq);
            xv[u].w[2 * i] = q.x;
            xv[u].w[2 * i + 1] = q.y;
          }
        } else {
          xv[u] = load32<false>(xr + k0 + u * 128, a.K - (k0 + u * 128 + kq), a.wide);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < MG; ++i)
#pragma unroll
          for (int p = 0; p < 8; p += 2)
            mma_s8(acc[i][nt], wv[u][i][0].w[p], wv[u][i][1].w[p], wv[u][i][0].w[p + 1], wv[u][i][1].w[p + 1], xv[u].w[p],
                   xv[u].w[p + 1]);
    }
    if (k0 + ROUND < a.K) load_w(k0 + ROUND);
  }
#pragma unroll
  for (int i = 0; i < MG; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 4; ++r) red[warp][i][nt][r][lane] = acc[i][nt][r];
  __syncthreads();
  // sixteen threads write the sixteen columns of a token
#pragma unroll
  for (int q = 0; q < NE; ++q) {
    const int e = threadIdx.x + q * 32 * WARPS, ch = e & 15, m = e >> 4, n = n0 + ch;
    if (m >= a.M || n >= a.N || m >= 8 * NT) continue;
    // where the product left column ch and token m: lane (ch % 8) * 4 + m % 8 / 2, register ch / 8 * 2 + m % 2
    const int l = (ch & 7) * 4 + ((m & 7) >> 1), r = (ch >> 3) * 2 + (m & 1), nt = m >> 3;
    float z[MG];
#pragma unroll
    for (int i = 0; i < MG; ++i) {
      int s = 0;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) s += red[w][i][nt][r][l];
      z[i] = fmaf(__int2float_rn(s), xs[q] * ws[q][i], bi[q][i]);
    }
    bf16* y = a.out + static_cast<size_t>(m) * a.N + n;
    float v = z[0];
    if (EPI == EPI_GELU) v = lo_f32(gelu_exp2(pack_f32x2(v, 0.f)));
    if (EPI == EPI_RESID) v += __bfloat162float(*y);
    if (GLU) v = lo_f32(silu_mul2(pack_f32x2(z[0], 0.f), pack_f32x2(z[MG - 1], 0.f)));
    *y = __float2bfloat16_rn(v);
  }
}

}  // namespace ts
