// rowops.cuh -- memory-bound row kernels: LayerNorm, the w-bar blend / merge, the
// tile gather of the stack input, per-row e4m3 quantisation, and the fp32 path's
// QK-RMSNorm + RoPE.  One warp per row, 16-byte vector accesses, fp32 arithmetic.
#pragma once

#include "common.cuh"

namespace ts {

// ---------------------------------------------------------------------------
// element access: bf16 or fp32 rows, 16-byte vectors (8 bf16 / 4 fp32)
// ---------------------------------------------------------------------------
template <typename T>
struct Vec;
template <>
struct Vec<bf16> {
  static constexpr int E = 8;
  __device__ static void load(const bf16* p, float* f) { bf16x8_to_f32(*reinterpret_cast<const uint4*>(p), f); }
  __device__ static void store(bf16* p, const float* f) { *reinterpret_cast<uint4*>(p) = f32_to_bf16x8(f); }
};
template <>
struct Vec<float> {
  static constexpr int E = 4;
  __device__ static void load(const float* p, float* f) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  }
  __device__ static void store(float* p, const float* f) { *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]); }
};

// Write one row held by a warp (NV vectors of E elements per lane, lane-strided) in
// the output format: T (bf16 / fp32), or e4m3 bytes + per-row scale absmax / 448, or
// signed 8-bit integers + per-row scale absmax / 127.
enum RowFormat : int { ROW_T = 0, ROW_E4M3 = 1, ROW_S8 = 2 };
template <typename T, int NV, int Q8>
__device__ __forceinline__ void store_row(const float (&v)[NV][Vec<T>::E], int lane, T* out, uint8_t* q8,
                                          float* qscale, size_t row, int d) {
  constexpr int E = Vec<T>::E;
  if (Q8 == ROW_T) {
#pragma unroll
    for (int i = 0; i < NV; ++i) Vec<T>::store(out + row * d + (i * 32 + lane) * E, v[i]);
  } else if (Q8 == ROW_S8) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) amax = max(amax, abs_bits(v[i][e]));
    const RowQuantS8 r = row_quant_s8(warp_max_u32(amax));
    if (lane == 0) qscale[row] = r.scale;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint32_t w[E / 4];
#pragma unroll
      for (int e = 0; e < E; e += 4) w[e / 4] = quant_s8x4(v[i][e], v[i][e + 1], v[i][e + 2], v[i][e + 3], r);
      uint8_t* dst = q8 + row * d + (i * 32 + lane) * E;
      if (E == 8)
        *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(w);
      else
        *reinterpret_cast<uint32_t*>(dst) = w[0];
    }
  } else {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) amax = fmaxf(amax, fabsf(v[i][e]));
    amax = warp_max(amax);
    const float s = amax > 0.f ? amax / 448.0f : 1.0f;
    const float inv = 1.0f / s;
    if (lane == 0) qscale[row] = s;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint16_t pk[E / 2];
#pragma unroll
      for (int e = 0; e < E; e += 2) pk[e / 2] = f32x2_to_e4m3x2(v[i][e] * inv, v[i][e + 1] * inv);
      uint8_t* dst = q8 + row * d + (i * 32 + lane) * E;
      if (E == 8)
        *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(pk);
      else
        *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(pk);
    }
  }
}

// ---------------------------------------------------------------------------
// LayerNorm (pre-LN block, [TileShare] Tab. S1 Norm1 / Norm2): population variance,
// two passes over the row held in registers.  NV = d / (32 * E) vectors per lane.
// With rms set it is RMSNorm (Tab. S6 "RMSNorm"): no centring and no bias.
// ---------------------------------------------------------------------------
// The first `row_blocks` blocks walk the rows grid-stride (one row per warp at a
// time, the warp's next row loaded before the current one is normalised, so two
// rows per warp are in flight); blocks past them (when rt.cs is set) fill the RoPE
// table that the next QKV GEMM reads.
template <typename T, int NV, int Q8>
__global__ void __launch_bounds__(256) layernorm_kernel(const T* __restrict__ x, int rows, int d,
                                                        const float* __restrict__ g, const float* __restrict__ b,
                                                        float eps, int rms, T* __restrict__ y, uint8_t* __restrict__ q8,
                                                        float* __restrict__ qscale, const RopeTable rt,
                                                        unsigned row_blocks) {
  pdl_wait();
  pdl_trigger();
  constexpr int E = Vec<T>::E;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x >= row_blocks) {
    rope_table_fill(rt, static_cast<int>((blockIdx.x - row_blocks) * blockDim.x + threadIdx.x));
    return;
  }
  const size_t step = static_cast<size_t>(row_blocks) * (blockDim.x >> 5);
  size_t row = static_cast<size_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  // the next row waits in registers as raw 16-byte vectors
  uint4 nx[NV];
  if (row < static_cast<size_t>(rows)) {
#pragma unroll
    for (int i = 0; i < NV; ++i) nx[i] = *reinterpret_cast<const uint4*>(x + row * d + (i * 32 + lane) * E);
  }
  for (; row < static_cast<size_t>(rows); row += step) {
    float v[NV][E];
#pragma unroll
    for (int i = 0; i < NV; ++i) Vec<T>::load(reinterpret_cast<const T*>(&nx[i]), v[i]);
    if (row + step < static_cast<size_t>(rows)) {
#pragma unroll
      for (int i = 0; i < NV; ++i) nx[i] = *reinterpret_cast<const uint4*>(x + (row + step) * d + (i * 32 + lane) * E);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) s += v[i][e];
    const float mean = rms ? 0.f : warp_sum(s) / d;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float c = v[i][e] - mean;
        q = fmaf(c, c, q);
      }
    const float rstd = rsqrtf(warp_sum(q) / d + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c0 = (i * 32 + lane) * E;
#pragma unroll
      for (int e = 0; e < E; e += 4) {   // gains and biases as 16-byte vectors
        const float4 gg = __ldg(reinterpret_cast<const float4*>(g + c0 + e));
        const float4 bb = rms ? make_float4(0.f, 0.f, 0.f, 0.f) : __ldg(reinterpret_cast<const float4*>(b + c0 + e));
        v[i][e] = (v[i][e] - mean) * rstd * gg.x + bb.x;
        v[i][e + 1] = (v[i][e + 1] - mean) * rstd * gg.y + bb.y;
        v[i][e + 2] = (v[i][e + 2] - mean) * rstd * gg.z + bb.z;
        v[i][e + 3] = (v[i][e + 3] - mean) * rstd * gg.w + bb.w;
      }
    }
    store_row<T, NV, Q8>(v, lane, y, q8, qscale, row, d);
  }
}

// generic fallback: any d (one warp per row, scalar, two passes over global memory)
template <typename T>
__global__ void __launch_bounds__(256) layernorm_generic_kernel(const T* __restrict__ x, int rows, int d,
                                                                const float* __restrict__ g,
                                                                const float* __restrict__ b, float eps, int rms,
                                                                T* __restrict__ y) {
  const int lane = threadIdx.x & 31;
  const size_t row = static_cast<size_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= static_cast<size_t>(rows)) return;
  const T* xr = x + row * d;
  float s = 0.f;
  for (int c = lane; c < d; c += 32) s += static_cast<float>(xr[c]);
  const float mean = rms ? 0.f : warp_sum(s) / d;
  float q = 0.f;
  for (int c = lane; c < d; c += 32) {
    const float t = static_cast<float>(xr[c]) - mean;
    q = fmaf(t, t, q);
  }
  const float rstd = rsqrtf(warp_sum(q) / d + eps);
  for (int c = lane; c < d; c += 32)
    y[row * d + c] = static_cast<T>((static_cast<float>(xr[c]) - mean) * rstd * g[c] + (rms ? 0.f : b[c]));
}

// ---------------------------------------------------------------------------
// The seam between two halves of a block, one pass over the residual stream:
//   x' = x + gate[group(r)] * scale * Norm_post(y),   xn = Norm_pre(x')
// with either norm, the gate and the scale optional.  Both norms are LayerNorm
// (population variance, two passes over the row in registers) or, with rms set,
// RMSNorm.  x' enters the second norm unrounded.
//
// Bound by DRAM: a row of x and of y read, of x' and of xn written.  What keeps a kernel
// from that bound is the work beside the bytes, so it is shared by as many columns as
// registers allow: a team of one warp (two for wide rows, more where only that divides
// the row) takes two rows at a time, NV 16-byte vectors of each in a thread, and each
// reduction, barrier and read of the gains and biases in shared memory serves both rows.
// Rows arrive by bulk copy without registers; the copy of a team's next y starts when
// this one is in registers, that of its next x when x' is formed (a deeper queue was no
// faster: the block's other teams fill the waits).
// ---------------------------------------------------------------------------
struct NormGateArgs {
  int rows, d, groups, rms;
  float eps;
  const float* post_g;     // [d] or null: y enters as it is
  const float* post_b;     // [d], LayerNorm only
  const float* pre_g;      // [d] or null: xn is not written
  const float* pre_b;      // [d], LayerNorm only
  const float* gate;       // [groups, d] or null: 1
  const float* scale;      // [d] or null: 1
  const int* row_group;    // [rows] or null: group 0
};

// group of a row; a number outside [0, groups) sets the device status and gives -1,
// and the row's outputs are left as they are
__device__ __forceinline__ int norm_gate_group(const NormGateArgs& a, size_t row) {
  if (!a.row_group) return 0;
  const int g = a.row_group[row];
  if (static_cast<unsigned>(g) >= static_cast<unsigned>(a.groups)) {
    set_status(kStatusDeviceCheck);
    return -1;
  }
  return g;
}

// E values in 16 bytes as packed pairs, and back
template <typename T>
__device__ __forceinline__ void unpack_pairs(const uint4& u, uint64_t (&p)[Vec<T>::E / 2]);
template <>
__device__ __forceinline__ void unpack_pairs<bf16>(const uint4& u, uint64_t (&p)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = pack_f32x2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
template <>
__device__ __forceinline__ void unpack_pairs<float>(const uint4& u, uint64_t (&p)[2]) {
  p[0] = pack_f32x2(__uint_as_float(u.x), __uint_as_float(u.y));
  p[1] = pack_f32x2(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ uint4 pack_pairs(const uint64_t (&p)[4]) {
  return make_uint4(pack_bf16(lo_f32(p[0]), hi_f32(p[0])), pack_bf16(lo_f32(p[1]), hi_f32(p[1])),
                    pack_bf16(lo_f32(p[2]), hi_f32(p[2])), pack_bf16(lo_f32(p[3]), hi_f32(p[3])));
}
__device__ __forceinline__ uint4 pack_pairs(const uint64_t (&p)[2]) {
  return make_uint4(__float_as_uint(lo_f32(p[0])), __float_as_uint(hi_f32(p[0])), __float_as_uint(lo_f32(p[1])),
                    __float_as_uint(hi_f32(p[1])));
}
// A row's 8-bit form from its largest magnitude (as bits), and the bytes of 2 P values held as pairs.
template <int Q8>
struct RowCode {
  RowQuantS8 s8;
  float e_scale, e_inv;
  __device__ __forceinline__ explicit RowCode(uint32_t amax) {
    if (Q8 == ROW_S8) {
      s8 = row_quant_s8(amax);
    } else {
      const float m = __uint_as_float(amax);
      e_scale = m > 0.f ? m / 448.0f : 1.0f;
      e_inv = 1.0f / e_scale;
    }
  }
  __device__ __forceinline__ float scale() const { return Q8 == ROW_S8 ? s8.scale : e_scale; }
  template <int P>
  __device__ __forceinline__ void put(const uint64_t (&v)[P], uint8_t* dst) const {
    uint32_t w[P / 2];
#pragma unroll
    for (int j = 0; j < P / 2; ++j) {
      const uint64_t p = v[2 * j], q = v[2 * j + 1];
      if (Q8 == ROW_S8)
        w[j] = quant_s8x4(lo_f32(p), hi_f32(p), lo_f32(q), hi_f32(q), s8);
      else
        w[j] = f32x2_to_e4m3x2(lo_f32(p) * e_inv, hi_f32(p) * e_inv) |
               (static_cast<uint32_t>(f32x2_to_e4m3x2(lo_f32(q) * e_inv, hi_f32(q) * e_inv)) << 16);
    }
    if (P == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[P / 2 - 1]);
    else
      *reinterpret_cast<uint32_t*>(dst) = w[0];
  }
};

// Few rows: a block of d / E threads (E columns each) takes two rows at a time, with its
// columns' gains, biases and gates in registers; what counts is the chain of loads and
// reductions of one pair.  In a graph 1 x 1536 takes 2.8 us against 6.3 by norm_gate_kernel,
// 512 x 1536 4.0 against 6.3 us; from about two pairs a block on the latter is faster
// (4000 x 1536: 16.7 us against 20.4).  Near the border the two lie within a fifth of each
// other, either way (2000 x 1024 8.2 and 8.1 us, 6000 x 256 7.3 and 6.1, 2000 x 2048 14.7
// and 16.4), as each goes up in steps of whole rounds of its grid.
template <typename T, int Q8>
__global__ void __launch_bounds__(256) norm_gate_few_kernel(const T* x, const T* y, T* x_out, T* xn, uint8_t* q8,
                                                            float* qscale, const NormGateArgs a) {
  __shared__ __align__(16) float red[2][2][8];
  constexpr int E = Vec<T>::E, P = E / 2;
  constexpr bool RAGGED = sizeof(T) == 4;    // fp32 rows may end inside a warp: threads behind the end hold zeros
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = threadIdx.x * E;
  const bool in = !RAGGED || c0 < a.d;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  if (threadIdx.x < 32) (&red[0][0][0])[threadIdx.x] = 0.f;    // warps that a block lacks add nothing
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  auto pairs_of = [&](const float* v, float fill, uint64_t (&p)[P]) {   // this thread's columns of a vector
#pragma unroll
    for (int i = 0; i < P; i += 2) {
      const float4 f = v && in ? __ldg(reinterpret_cast<const float4*>(v + c0 + 2 * i)) : make_float4(fill, fill, fill, fill);
      p[i] = pack_f32x2(f.x, f.y);
      p[i + 1] = pack_f32x2(f.z, f.w);
    }
  };
  uint64_t post_g[P], post_b[P], pre_g[P], pre_b[P], scale[P], gs[P];
  pairs_of(a.post_g, 1.f, post_g);
  pairs_of(a.rms ? nullptr : a.post_b, 0.f, post_b);
  pairs_of(a.pre_g, 1.f, pre_g);
  pairs_of(a.rms ? nullptr : a.pre_b, 0.f, pre_b);
  pairs_of(a.scale, 1.f, scale);
  int gs_group = -1;
  auto load_gate = [&](int group) {        // gate * scale of a group
    pairs_of(a.gate ? a.gate + static_cast<size_t>(group) * a.d : nullptr, 1.f, gs);
#pragma unroll
    for (int i = 0; i < P; ++i) gs[i] = mul_f32x2(gs[i], scale[i]);
    gs_group = group;
  };
  int rb = 0;                              // reduction buffer: a buffer's next use is two barriers away
  auto sum2 = [&](float& s0, float& s1) {  // (s0, s1) of every thread -> their sums over the block
    float m = lane < 16 ? s0 : s1;
    m += __shfl_xor_sync(0xffffffffu, lane < 16 ? s1 : s0, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    if ((lane & 15) == 0) red[rb][lane >> 4][warp] = m;
    __syncthreads();
    const float4* r = reinterpret_cast<const float4*>(&red[rb][0][0]);
    const float4 a0 = r[0], a1 = r[1], b0 = r[2], b1 = r[3];
    s0 = ((a0.x + a0.y) + (a0.z + a0.w)) + ((a1.x + a1.y) + (a1.z + a1.w));
    s1 = ((b0.x + b0.y) + (b0.z + b0.w)) + ((b1.x + b1.y) + (b1.z + b1.w));
    rb ^= 1;
  };
  auto max2 = [&](uint32_t& s0, uint32_t& s1) {
    s0 = warp_max_u32(s0);
    s1 = warp_max_u32(s1);
    if (lane == 0) {
      red[rb][0][warp] = __uint_as_float(s0);
      red[rb][1][warp] = __uint_as_float(s1);
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      s0 = max(s0, __float_as_uint(red[rb][0][w]));
      s1 = max(s1, __float_as_uint(red[rb][1][w]));
    }
    rb ^= 1;
  };
  auto norm2 = [&](uint64_t (&v0)[P], uint64_t (&v1)[P], const uint64_t (&g)[P], const uint64_t (&b)[P]) {
    if (!a.rms) {
      uint64_t t0 = 0ull, t1 = 0ull;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        t0 = add_f32x2(t0, v0[i]);
        t1 = add_f32x2(t1, v1[i]);
      }
      float s0 = lo_f32(t0) + hi_f32(t0), s1 = lo_f32(t1) + hi_f32(t1);
      sum2(s0, s1);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        v0[i] = in ? add_f32x2(v0[i], splat_f32x2(-s0 * inv_d)) : 0ull;
        v1[i] = in ? add_f32x2(v1[i], splat_f32x2(-s1 * inv_d)) : 0ull;
      }
    }
    uint64_t t0 = 0ull, t1 = 0ull;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      t0 = fma_f32x2(v0[i], v0[i], t0);
      t1 = fma_f32x2(v1[i], v1[i], t1);
    }
    float q0 = lo_f32(t0) + hi_f32(t0), q1 = lo_f32(t1) + hi_f32(t1);
    sum2(q0, q1);
    const uint64_t r0 = splat_f32x2(rsqrtf(q0 * inv_d + a.eps)), r1 = splat_f32x2(rsqrtf(q1 * inv_d + a.eps));
#pragma unroll
    for (int i = 0; i < P; ++i) {
      v0[i] = fma_f32x2(mul_f32x2(v0[i], r0), g[i], b[i]);
      v1[i] = fma_f32x2(mul_f32x2(v1[i], r1), g[i], b[i]);
    }
  };
  const size_t rows = a.rows;
  for (size_t row = 2 * static_cast<size_t>(blockIdx.x); row < rows; row += 2 * static_cast<size_t>(gridDim.x)) {
    const bool two = row + 1 < rows;
    const size_t o0 = row * a.d + c0, o1 = two ? o0 + a.d : o0;
    uint64_t x0[P], x1[P], v0[P], v1[P];
    const uint4 zero = make_uint4(0, 0, 0, 0);
    unpack_pairs<T>(in ? *reinterpret_cast<const uint4*>(y + o0) : zero, v0);
    unpack_pairs<T>(in ? *reinterpret_cast<const uint4*>(y + o1) : zero, v1);
    unpack_pairs<T>(in ? *reinterpret_cast<const uint4*>(x + o0) : zero, x0);
    unpack_pairs<T>(in ? *reinterpret_cast<const uint4*>(x + o1) : zero, x1);
    const int g0 = norm_gate_group(a, row), g1 = two ? norm_gate_group(a, row + 1) : -1;
    if (g0 >= 0 && g0 != gs_group) load_gate(g0);
    if (a.post_g) norm2(v0, v1, post_g, post_b);
#pragma unroll
    for (int i = 0; i < P; ++i) v0[i] = fma_f32x2(gs[i], v0[i], x0[i]);
    if (g1 >= 0 && g1 != gs_group) load_gate(g1);
#pragma unroll
    for (int i = 0; i < P; ++i) v1[i] = fma_f32x2(gs[i], v1[i], x1[i]);
    if (g0 >= 0 && in) *reinterpret_cast<uint4*>(x_out + o0) = pack_pairs(v0);
    if (g1 >= 0 && in) *reinterpret_cast<uint4*>(x_out + o1) = pack_pairs(v1);
    if (!a.pre_g) continue;
    if (!in) {
#pragma unroll
      for (int i = 0; i < P; ++i) v0[i] = v1[i] = 0ull;
    }
    norm2(v0, v1, pre_g, pre_b);
    if (Q8 == ROW_T) {
      if (g0 >= 0 && in) *reinterpret_cast<uint4*>(xn + o0) = pack_pairs(v0);
      if (g1 >= 0 && in) *reinterpret_cast<uint4*>(xn + o1) = pack_pairs(v1);
    } else {
      uint32_t m0 = 0, m1 = 0;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        m0 = max(m0, max(abs_bits(lo_f32(v0[i])), abs_bits(hi_f32(v0[i]))));
        m1 = max(m1, max(abs_bits(lo_f32(v1[i])), abs_bits(hi_f32(v1[i]))));
      }
      max2(m0, m1);
      const RowCode<Q8> r0(m0), r1(m1);
      if (g0 >= 0) {
        if (threadIdx.x == 0) qscale[row] = r0.scale();
        r0.template put<P>(v0, q8 + o0);
      }
      if (g1 >= 0) {
        if (threadIdx.x == 0) qscale[row + 1] = r1.scale();
        r1.template put<P>(v1, q8 + o1);
      }
    }
  }
}

constexpr int kNormGateTeamWarps = 8;    // most warps of a team
constexpr int kNormGateTeams = 32;       // most teams of a block
// most threads of a block by the registers that NV vectors of two rows take (fp32 vectors take half as many, but more
// warps a block were slower there: 20000 x 1024 68 us with 640 threads, 55 with 384)
template <int NV>
constexpr int norm_gate_threads() {
  return NV == 1 ? 896 : NV == 2 ? 640 : NV == 3 ? 512 : 384;
}

template <typename T, int NV, int Q8>
__global__ void __launch_bounds__(norm_gate_threads<NV>(), 1)
    norm_gate_kernel(const T* x, const T* y, T* x_out, T* xn, uint8_t* q8, float* qscale, const NormGateArgs a,
                     int team_warps) {
  extern __shared__ __align__(128) uint8_t smem[];    // vectors [4][d], then per team two rows of y and two of x
  __shared__ __align__(16) float red[kNormGateTeams][2][2][kNormGateTeamWarps];
  __shared__ __align__(8) uint64_t bars[kNormGateTeams][2];    // y, x
  constexpr int E = Vec<T>::E, P = E / 2, Q = E / 4;
  constexpr bool RAGGED = sizeof(T) == 4;    // fp32 rows may end inside a team's vectors: what lies behind is zero
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % team_warps, team = (threadIdx.x >> 5) / team_warps;
  const int tsize = 32 * team_warps, t = threadIdx.x - team * tsize, teams = blockDim.x / tsize;
  const uint32_t rowbytes = static_cast<uint32_t>(a.d) * sizeof(T);
  const float inv_d = 1.0f / static_cast<float>(a.d);
  const int quads = RAGGED ? NV * Q * tsize : a.d / 4;    // four-column quads of a vector in shared memory
  auto in = [&](int i) -> bool { return !RAGGED || (i * tsize + t) * E < a.d; };
  uint8_t* ring = smem + static_cast<size_t>(64) * quads + static_cast<size_t>(team) * 4 * rowbytes;
  if (t == 0) {
    mbar_init(smem_u32(&bars[team][0]), 1);
    mbar_init(smem_u32(&bars[team][1]), 1);
    fence_barrier_init();
  }
  if (t < 32) (&red[team][0][0][0])[t] = 0.f;    // warps that a team lacks add nothing
  // whether a flag holds in all threads of the team, and a barrier of them
  auto team_all = [&](bool f) -> bool {
    if (team_warps == 1) return __all_sync(0xffffffffu, f);
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"(f ? 1u : 0u), "r"(1 + team), "r"(tsize)
        : "memory");
    return r != 0;
  };
  team_all(true);
  pdl_wait();
  pdl_trigger();
  const size_t rows = a.rows, step = 2 * static_cast<size_t>(gridDim.x) * teams;
  size_t row = 2 * (static_cast<size_t>(blockIdx.x) * teams + team);
  // copy of a pair of rows of y (k = 0) or x (k = 1), by one thread of the team
  auto issue = [&](int k, size_t r) {
    const uint32_t n = r + 1 < rows ? 2 * rowbytes : rowbytes, bar = smem_u32(&bars[team][k]);
    mbar_expect_tx(bar, n);
    bulk_load(smem_u32(ring) + static_cast<uint32_t>(2 * k) * rowbytes, (k ? x : y) + r * a.d, n, bar);
  };
  if (t == 0 && row < rows) {
    issue(0, row);
    issue(1, row);
  }
  // The shared vectors.  Thread t owns vectors i * tsize + t of a row; the four-column quads of a vector lie tsize
  // float4s apart, so that a warp reads them without bank conflicts.
  const float* src[4] = {a.post_g, a.rms ? nullptr : a.post_b, a.pre_g, a.rms ? nullptr : a.pre_b};
  float4* vecs = reinterpret_cast<float4*>(smem);
  for (int m0 = team; m0 < 4 * NV * Q; m0 += 8 * teams) {      // the teams take turns, eight loads in flight
    float4 f[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int m = m0 + u * teams, k = m / (NV * Q), c = m % (NV * Q);
      const float* v = k == 0 ? src[0] : k == 1 ? src[1] : k == 2 ? src[2] : src[3];
      f[u] = m < 4 * NV * Q && v && in(c / Q) ? __ldg(reinterpret_cast<const float4*>(v) + (c / Q * tsize + t) * Q + c % Q)
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int m = m0 + u * teams;
      if (m < 4 * NV * Q) vecs[m / (NV * Q) * quads + m % (NV * Q) * tsize + t] = f[u];
    }
  }
  uint64_t gs[NV][P];                      // gate * scale of this thread's columns, for the group gs_group
  int gs_group = -1;
  auto load_gate = [&](int group) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < Q; ++j) {
        const size_t c = static_cast<size_t>(i * tsize + t) * E + 4 * j;
        float4 f = make_float4(1.f, 1.f, 1.f, 1.f);
        if (a.gate && in(i)) f = __ldg(reinterpret_cast<const float4*>(a.gate + static_cast<size_t>(group) * a.d + c));
        if (a.scale && in(i)) {
          const float4 sc = __ldg(reinterpret_cast<const float4*>(a.scale + c));
          f.x *= sc.x; f.y *= sc.y; f.z *= sc.z; f.w *= sc.w;
        }
        gs[i][2 * j] = pack_f32x2(f.x, f.y);
        gs[i][2 * j + 1] = pack_f32x2(f.z, f.w);
      }
    gs_group = group;
  };
  if (row < rows) {
    const int g = norm_gate_group(a, row);
    if (g >= 0) load_gate(g);
  }
  __syncthreads();
  int rb = 0;                              // reduction buffer: a buffer's next use is two barriers away
  // (s0, s1) of every thread -> their sums over the team; returns `flag` as team_all gives it
  auto sum2 = [&](float& s0, float& s1, bool flag) -> bool {
    float m = lane < 16 ? s0 : s1;
    m += __shfl_xor_sync(0xffffffffu, lane < 16 ? s1 : s0, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    if (team_warps == 1) {
      const float other = __shfl_xor_sync(0xffffffffu, m, 16);
      s0 = lane < 16 ? m : other;
      s1 = lane < 16 ? other : m;
      return __all_sync(0xffffffffu, flag);
    }
    if ((lane & 15) == 0) red[team][rb][lane >> 4][warp] = m;
    const bool all = team_all(flag);
    const float4* r = reinterpret_cast<const float4*>(&red[team][rb][0][0]);
    const float4 a0 = r[0], a1 = r[1], b0 = r[2], b1 = r[3];
    s0 = ((a0.x + a0.y) + (a0.z + a0.w)) + ((a1.x + a1.y) + (a1.z + a1.w));
    s1 = ((b0.x + b0.y) + (b0.z + b0.w)) + ((b1.x + b1.y) + (b1.z + b1.w));
    rb ^= 1;
    return all;
  };
  auto max2 = [&](uint32_t& s0, uint32_t& s1) {
    s0 = warp_max_u32(s0);
    s1 = warp_max_u32(s1);
    if (team_warps == 1) return;
    if (lane == 0) {
      red[team][rb][0][warp] = __uint_as_float(s0);
      red[team][rb][1][warp] = __uint_as_float(s1);
    }
    team_all(true);
    const uint4* r = reinterpret_cast<const uint4*>(&red[team][rb][0][0]);
    const uint4 a0 = r[0], a1 = r[1], b0 = r[2], b1 = r[3];
    s0 = max(max(max(a0.x, a0.y), max(a0.z, a0.w)), max(max(a1.x, a1.y), max(a1.z, a1.w)));
    s1 = max(max(max(b0.x, b0.y), max(b0.z, b0.w)), max(max(b1.x, b1.y), max(b1.z, b1.w)));
    rb ^= 1;
  };
  typedef uint64_t Row[NV][P];
  auto total = [&](const Row& v) -> float {
    uint64_t u = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int p = 0; p < P; p += 2) u = add_f32x2(u, add_f32x2(v[i][p], v[i][p + 1]));
    return lo_f32(u) + hi_f32(u);
  };
  auto squares = [&](const Row& v) -> float {
    uint64_t u = 0ull, w = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int p = 0; p < P; p += 2) {
        u = fma_f32x2(v[i][p], v[i][p], u);
        w = fma_f32x2(v[i][p + 1], v[i][p + 1], w);
      }
    u = add_f32x2(u, w);
    return lo_f32(u) + hi_f32(u);
  };
  // both rows: v -> (v - mean) * rstd * g + b with g, b the shared vectors k, k + 1; the last barrier carries `flag`
  auto norm2 = [&](Row& v0, Row& v1, int k, bool flag) -> bool {
    if (!a.rms) {
      float s0 = total(v0), s1 = total(v1);
      sum2(s0, s1, true);
      const uint64_t m0 = splat_f32x2(-s0 * inv_d), m1 = splat_f32x2(-s1 * inv_d);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int p = 0; p < P; ++p) {
          v0[i][p] = in(i) ? add_f32x2(v0[i][p], m0) : 0ull;
          v1[i][p] = in(i) ? add_f32x2(v1[i][p], m1) : 0ull;
        }
    }
    float q0 = squares(v0), q1 = squares(v1);
    const bool all = sum2(q0, q1, flag);
    const uint64_t r0 = splat_f32x2(rsqrtf(q0 * inv_d + a.eps)), r1 = splat_f32x2(rsqrtf(q1 * inv_d + a.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < Q; ++j) {
        const float4 g = vecs[k * quads + (i * Q + j) * tsize + t], b = vecs[(k + 1) * quads + (i * Q + j) * tsize + t];
        const uint64_t g0 = pack_f32x2(g.x, g.y), g1 = pack_f32x2(g.z, g.w), b0 = pack_f32x2(b.x, b.y),
                       b1 = pack_f32x2(b.z, b.w);
        v0[i][2 * j] = fma_f32x2(mul_f32x2(v0[i][2 * j], r0), g0, b0);
        v1[i][2 * j] = fma_f32x2(mul_f32x2(v1[i][2 * j], r1), g0, b0);
        v0[i][2 * j + 1] = fma_f32x2(mul_f32x2(v0[i][2 * j + 1], r0), g1, b1);
        v1[i][2 * j + 1] = fma_f32x2(mul_f32x2(v1[i][2 * j + 1], r1), g1, b1);
      }
    return all;
  };
  auto put = [&](T* out, size_t r, const Row& v) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in(i)) *reinterpret_cast<uint4*>(out + r * a.d + static_cast<size_t>(i * tsize + t) * E) = pack_pairs(v[i]);
  };
  const uint8_t* ys = ring + t * 16;
  const uint8_t* xs = ys + 2 * static_cast<size_t>(rowbytes);
  uint32_t phase = 0;
  bool ok = true;
  for (; row < rows; row += step, phase ^= 1) {
    const int g0 = norm_gate_group(a, row), g1 = row + 1 < rows ? norm_gate_group(a, row + 1) : -1;
    const bool more = row + step < rows;
    // both copies are waited for here, so that one barrier tells the team whether either gave up
    const bool here = mbar_wait(smem_u32(&bars[team][0]), phase) && mbar_wait(smem_u32(&bars[team][1]), phase);
    Row v0, v1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint4 zero = make_uint4(0, 0, 0, 0);
      unpack_pairs<T>(in(i) ? *reinterpret_cast<const uint4*>(ys + i * tsize * 16) : zero, v0[i]);
      unpack_pairs<T>(in(i) ? *reinterpret_cast<const uint4*>(ys + rowbytes + i * tsize * 16) : zero, v1[i]);
    }
    fence_proxy_async_smem();
    ok = team_all(here);                   // and every thread has read y
    if (!ok) break;
    if (more && t == 0) issue(0, row + step);
    if (a.post_g) norm2(v0, v1, 0, true);
    if (g0 >= 0 && g0 != gs_group) load_gate(g0);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint64_t r[P];
      unpack_pairs<T>(in(i) ? *reinterpret_cast<const uint4*>(xs + i * tsize * 16) : make_uint4(0, 0, 0, 0), r);
#pragma unroll
      for (int p = 0; p < P; ++p) v0[i][p] = fma_f32x2(gs[i][p], v0[i][p], r[p]);
    }
    if (g1 >= 0 && g1 != gs_group) load_gate(g1);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint64_t r[P];
      unpack_pairs<T>(in(i) ? *reinterpret_cast<const uint4*>(xs + rowbytes + i * tsize * 16) : make_uint4(0, 0, 0, 0), r);
#pragma unroll
      for (int p = 0; p < P; ++p) v1[i][p] = fma_f32x2(gs[i][p], v1[i][p], r[p]);
    }
    fence_proxy_async_smem();
    team_all(true);                        // every thread has read x
    if (more && t == 0) issue(1, row + step);
    if (g0 >= 0) put(x_out, row, v0);
    if (g1 >= 0) put(x_out, row + 1, v1);
    if (a.pre_g) {
      // (behind the end of a ragged row x' is zero here, as y, x and the vectors are)
      norm2(v0, v1, 2, true);
      if (Q8 == ROW_T) {
        if (g0 >= 0) put(xn, row, v0);
        if (g1 >= 0) put(xn, row + 1, v1);
      } else {
        uint32_t m0 = 0, m1 = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int p = 0; p < P; ++p) {
            m0 = max(m0, max(abs_bits(lo_f32(v0[i][p])), abs_bits(hi_f32(v0[i][p]))));
            m1 = max(m1, max(abs_bits(lo_f32(v1[i][p])), abs_bits(hi_f32(v1[i][p]))));
          }
        max2(m0, m1);
        auto put8 = [&](size_t r, const Row& v, uint32_t amax) {
          const RowCode<Q8> code(amax);
          if (t == 0) qscale[r] = code.scale();
#pragma unroll
          for (int i = 0; i < NV; ++i) code.template put<P>(v[i], q8 + r * a.d + static_cast<size_t>(i * tsize + t) * E);
        };
        if (g0 >= 0) put8(row, v0, m0);
        if (g1 >= 0) put8(row + 1, v1, m1);
      }
    }
  }
  // no copy may still be landing when the block exits (matters only after a timeout)
  if (!ok) {
    mbar_wait(smem_u32(&bars[team][0]), phase);
    mbar_wait(smem_u32(&bars[team][1]), phase);
  }
}

// fp32 rows wider than a team: one warp per row, scalar.  Only the lane that holds a column
// reads or writes it, so x' may replace x and serves as the row's storage between
// the two norms.
__global__ void __launch_bounds__(256) norm_gate_generic_kernel(const float* x, const float* y, float* x_out, float* xn,
                                                                const NormGateArgs a) {
  const int lane = threadIdx.x & 31;
  const size_t row = static_cast<size_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= static_cast<size_t>(a.rows)) return;
  const int group = norm_gate_group(a, row);
  if (group < 0) return;
  auto stats = [&](const float* v, float& mean, float& rstd) {
    float s = 0.f, q = 0.f;
    for (int c = lane; c < a.d; c += 32) s += v[c];
    mean = a.rms ? 0.f : warp_sum(s) / a.d;
    for (int c = lane; c < a.d; c += 32) {
      const float t = v[c] - mean;
      q = fmaf(t, t, q);
    }
    rstd = rsqrtf(warp_sum(q) / a.d + a.eps);
  };
  const size_t off = row * a.d;
  const float* gate = a.gate ? a.gate + static_cast<size_t>(group) * a.d : nullptr;
  float mean = 0.f, rstd = 1.f;
  if (a.post_g) stats(y + off, mean, rstd);
  for (int c = lane; c < a.d; c += 32) {
    float v = y[off + c];
    if (a.post_g) v = (v - mean) * rstd * a.post_g[c] + (a.rms ? 0.f : a.post_b[c]);
    x_out[off + c] = fmaf((gate ? gate[c] : 1.f) * (a.scale ? a.scale[c] : 1.f), v, x[off + c]);
  }
  if (!a.pre_g) return;
  stats(x_out + off, mean, rstd);
  for (int c = lane; c < a.d; c += 32)
    xn[off + c] = (x_out[off + c] - mean) * rstd * a.pre_g[c] + (a.rms ? 0.f : a.pre_b[c]);
}

// ---------------------------------------------------------------------------
// Blend / merge ([TileShare] Fig. 2: overlap tokens' attention outputs blended with
// w-bar; Fig. 3b: per-tile states merged).  Row u < U: fp32 sum over the token's
// CSR entries in ascending tile order of wbar * P[ent]; row U + t*R + i: P[t*N + i].  One
// warp writes each output row once; no atomics, so the result is deterministic.
// ---------------------------------------------------------------------------
template <typename T, int NV, int Q8>
__global__ void __launch_bounds__(256) merge_kernel(const T* __restrict__ P, int rows, int U, int N, int R, int d,
                                                    const int* __restrict__ tok_ptr, const int* __restrict__ tok_ent,
                                                    const float* __restrict__ wbar, T* __restrict__ A,
                                                    uint8_t* __restrict__ q8, float* __restrict__ qscale) {
  pdl_wait();
  pdl_trigger();
  constexpr int E = Vec<T>::E;
  const int lane = threadIdx.x & 31;
  const size_t row = static_cast<size_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= static_cast<size_t>(rows)) return;
  float v[NV][E];
  if (row < static_cast<size_t>(U)) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] = 0.f;
    const int e0 = __ldg(tok_ptr + row), e1 = __ldg(tok_ptr + row + 1);
    for (int e = e0; e < e1; ++e) {
      const float w = __ldg(wbar + e);
      const T* src = P + static_cast<size_t>(__ldg(tok_ent + e)) * d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[E];
        Vec<T>::load(src + (i * 32 + lane) * E, f);
#pragma unroll
        for (int k = 0; k < E; ++k) v[i][k] = fmaf(w, f[k], v[i][k]);
      }
    }
  } else {
    const size_t reg = row - U;   // register i of tile t: row t*N + i of P
    const T* src = P + ((reg / R) * static_cast<size_t>(N) + reg % R) * d;
#pragma unroll
    for (int i = 0; i < NV; ++i) Vec<T>::load(src + (i * 32 + lane) * E, v[i]);
  }
  store_row<T, NV, Q8>(v, lane, A, q8, qscale, row, d);
}

// The same blend with the tile rows staged in shared memory: each warp owns two
// buffers of `cover` rows (cover = most tiles on one token) and keeps two output
// rows in flight; for each, the lanes read the token's entries (one per lane) and
// issue one bulk copy per entry, so loads in flight hold no registers.  Row
// U + t*R + i is the single entry t*N + i with weight 1.  Sums run in ascending entry order,
// as in merge_kernel.
constexpr int kMergeWarps = 4;
template <typename T, int NV, int Q8>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_bulk_kernel(
    const T* __restrict__ P, int rows, int U, int N, int R, int d, const int* __restrict__ tok_ptr,
    const int* __restrict__ tok_ent, const float* __restrict__ wbar, int cover, T* __restrict__ A,
    uint8_t* __restrict__ q8, float* __restrict__ qscale) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int E = Vec<T>::E;
  const int lane = threadIdx.x & 31, wib = threadIdx.x >> 5;
  const uint32_t rowbytes = static_cast<uint32_t>(d) * sizeof(T);
  uint8_t* wbuf = smem + static_cast<size_t>(wib) * 2 * cover * rowbytes;
  const uint32_t bar = smem_u32(smem + static_cast<size_t>(kMergeWarps) * 2 * cover * rowbytes) + 16 * wib;
  if (lane == 0) {
    mbar_init(bar, 1);
    mbar_init(bar + 8, 1);
    fence_barrier_init();
  }
  __syncwarp();
  pdl_wait();
  pdl_trigger();
  // Row metadata runs ahead of the copies so that no dependent L2 round trip sits on
  // a row's path: lane k holds the CSR row pointer and entry count of this warp's
  // row base + k (refreshed every 32 rows), and the entries and weights of a row are
  // loaded one row before its copies are issued.  A register row U + t*R + i is
  // encoded as pointer -1 - (t*R + i), one entry t*N + i of weight 1.
  const int stride = gridDim.x * kMergeWarps;
  const int r0 = blockIdx.x * kMergeWarps + wib;
  int my_e0 = 0, my_n = 0;
  auto load_ptrs = [&](int base) {
    const int r = r0 + (base + lane) * stride;
    my_e0 = 0;
    my_n = 0;
    if (r < rows) {
      if (r < U) {
        my_e0 = __ldg(tok_ptr + r);
        my_n = __ldg(tok_ptr + r + 1) - my_e0;
      } else {
        my_e0 = -1 - (r - U);
        my_n = 1;
      }
    }
  };
  // entries (lane k < n: entry k and its weight) of this warp's i-th row
  auto load_ents = [&](int i, int& ent, float& wl, int& n) {
    const int e0 = __shfl_sync(0xffffffffu, my_e0, i & 31);
    n = __shfl_sync(0xffffffffu, my_n, i & 31);
    ent = 0;
    wl = 0.f;
    if (lane < n) {
      if (e0 >= 0) {
        ent = __ldg(tok_ent + e0 + lane);
        wl = __ldg(wbar + e0 + lane);
      } else {
        const int reg = -1 - e0;
        ent = (reg / R) * N + reg % R;
        wl = 1.f;
      }
    }
  };
  // copies of a row's entries into buffer b
  auto issue = [&](int b, int n, int ent) {
    fence_proxy_async_smem();   // this warp's reads of the buffer precede the copies that overwrite it
    __syncwarp();
    if (lane == 0) mbar_expect_tx(bar + 8 * b, n * rowbytes);
    __syncwarp();
    if (lane < n)
      bulk_load(smem_u32(wbuf + (static_cast<size_t>(b) * cover + lane) * rowbytes), P + static_cast<size_t>(ent) * d,
                rowbytes, bar + 8 * b);
  };
  int row = r0;
  int nc = 0, nn = 0, entc = 0, entn = 0;
  float wc = 0.f, wn = 0.f;
  bool pending_next = false;
  int broke_at = -1;
  load_ptrs(0);
  if (row < rows) {
    load_ents(0, entc, wc, nc);
    issue(0, nc, entc);
  }
  if (row + stride < rows) load_ents(1, entn, wn, nn);
  for (int i = 0; row < rows; ++i, row += stride) {
    pending_next = row + stride < rows;
    if (pending_next) issue((i + 1) & 1, nn, entn);
    int n2 = 0, ent2 = 0;
    float w2 = 0.f;
    if (row + 2 * stride < rows) {
      if (((i + 2) & 31) == 0) load_ptrs(i + 2);
      load_ents(i + 2, ent2, w2, n2);
    }
    if (!mbar_wait(bar + 8 * (i & 1), (i >> 1) & 1)) {
      broke_at = i;
      break;
    }
    pending_next = false;
    const uint8_t* buf = wbuf + static_cast<size_t>(i & 1) * cover * rowbytes;
    float v[NV][E];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) v[k][e] = 0.f;
    for (int k = 0; k < nc; ++k) {
      const float w = __shfl_sync(0xffffffffu, wc, k);
      const T* src = reinterpret_cast<const T*>(buf + static_cast<size_t>(k) * rowbytes);
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        float f[E];
        Vec<T>::load(src + (q * 32 + lane) * E, f);
#pragma unroll
        for (int e = 0; e < E; ++e) v[q][e] = fmaf(w, f[e], v[q][e]);
      }
    }
    store_row<T, NV, Q8>(v, lane, A, q8, qscale, row, d);
    nc = nn;
    wc = wn;
    nn = n2;
    entn = ent2;
    wn = w2;
  }
  // no copy may still be landing when the CTA exits (matters only after a timeout)
  if (broke_at >= 0) {
    mbar_wait(bar + 8 * (broke_at & 1), (broke_at >> 1) & 1);
    if (pending_next) mbar_wait(bar + 8 * ((broke_at + 1) & 1), ((broke_at + 1) >> 1) & 1);
  }
}

// generic fallback of the blend for any d (scalar)
template <typename T>
__global__ void __launch_bounds__(256) merge_generic_kernel(const T* __restrict__ P, int rows, int U, int N, int R, int d,
                                                            const int* __restrict__ tok_ptr,
                                                            const int* __restrict__ tok_ent,
                                                            const float* __restrict__ wbar, T* __restrict__ A) {
  const int lane = threadIdx.x & 31;
  const size_t row = static_cast<size_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= static_cast<size_t>(rows)) return;
  for (int c = lane; c < d; c += 32) {
    float acc = 0.f;
    if (row < static_cast<size_t>(U)) {
      for (int e = tok_ptr[row]; e < tok_ptr[row + 1]; ++e)
        acc = fmaf(wbar[e], static_cast<float>(P[static_cast<size_t>(tok_ent[e]) * d + c]), acc);
    } else {
      const size_t reg = row - U;
      acc = static_cast<float>(P[((reg / R) * static_cast<size_t>(N) + reg % R) * d + c]);
    }
    A[row * d + c] = static_cast<T>(acc);
  }
}

// ---------------------------------------------------------------------------
// Stack input: per-tile copies X[t*N + s] of grid tokens S0 and global tokens G0
// (row map of the shared layout: < U grid token, >= U global token).
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) gather_rows_kernel(const uint8_t* __restrict__ S0,
                                                          const uint8_t* __restrict__ G0,
                                                          const int* __restrict__ rowmap, int nrows, int U,
                                                          size_t row_bytes, uint8_t* __restrict__ X) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const size_t r = static_cast<size_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (r >= static_cast<size_t>(nrows)) return;
  const int src = __ldg(rowmap + r);
  const uint8_t* s = src < U ? S0 + static_cast<size_t>(src) * row_bytes : G0 + static_cast<size_t>(src - U) * row_bytes;
  for (size_t c = lane * 16; c < row_bytes; c += 32 * 16)
    *reinterpret_cast<uint4*>(X + r * row_bytes + c) = *reinterpret_cast<const uint4*>(s + c);
}

// ---------------------------------------------------------------------------
// Partial sharing ([TileShare] Tab. 1 top): a per-token result R [U + T, d] of a
// shared operation is added to every tile's copy of the token, X[r] += R[rowmap[r]]
// for the T * N per-tile rows (a tile's registers take its register rows of R).  fp32 add, one
// warp per row, 16-byte vectors; every X row is written by one warp.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) scatter_add_rows_kernel(const T* __restrict__ R, const int* __restrict__ rowmap,
                                                               int nrows, int d, T* __restrict__ X) {
  pdl_wait();
  pdl_trigger();
  constexpr int E = Vec<T>::E;
  const int lane = threadIdx.x & 31;
  const size_t r = static_cast<size_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (r >= static_cast<size_t>(nrows)) return;
  const T* src = R + static_cast<size_t>(__ldg(rowmap + r)) * d;
  T* dst = X + r * d;
  for (int c = lane * E; c < d; c += 32 * E) {
    float a[E], b[E];
    Vec<T>::load(dst + c, a);
    Vec<T>::load(src + c, b);
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] += b[e];
    Vec<T>::store(dst + c, a);
  }
}

// ---------------------------------------------------------------------------
// Per-row e4m3 quantisation of a bf16 matrix: scale = absmax / 448 (1 if zero),
// q = e4m3(x / scale), nearest-even, saturating.  cols % 8 == 0.
// ---------------------------------------------------------------------------
// Each lane walks its 16-byte vectors eight at a time (eight loads in flight, so
// the pass is not bound by one load's latency); the second pass reads the row again
// (from L1 / L2) to quantise it.
__global__ void __launch_bounds__(256) quantize_rows_kernel(const bf16* __restrict__ x, int rows, int cols,
                                                            uint8_t* __restrict__ q, float* __restrict__ scale) {
  pdl_wait();
  pdl_trigger();
  constexpr int U = 8;   // vectors in flight per lane
  const int lane = threadIdx.x & 31;
  const size_t row = static_cast<size_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= static_cast<size_t>(rows)) return;
  const bf16* xr = x + row * cols;
  float amax = 0.f;
  for (int c0 = lane * 8; c0 < cols; c0 += 256 * U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * 256 < cols) v[u] = *reinterpret_cast<const uint4*>(xr + c0 + u * 256);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * 256 < cols) {
        float f[8];
        bf16x8_to_f32(v[u], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
      }
  }
  amax = warp_max(amax);
  const float s = amax > 0.f ? amax / 448.0f : 1.0f;
  const float inv = 1.0f / s;   // one division per row; x / s becomes x * (1 / s) (within an fp32 ulp)
  if (lane == 0) scale[row] = s;
  for (int c0 = lane * 8; c0 < cols; c0 += 256 * U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * 256 < cols) v[u] = *reinterpret_cast<const uint4*>(xr + c0 + u * 256);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * 256 < cols) {
        float f[8];
        bf16x8_to_f32(v[u], f);
        uint16_t pk[4];
#pragma unroll
        for (int e = 0; e < 8; e += 2) pk[e / 2] = f32x2_to_e4m3x2(f[e] * inv, f[e + 1] * inv);
        *reinterpret_cast<uint2*>(q + row * cols + c0 + u * 256) = *reinterpret_cast<const uint2*>(pk);
      }
  }
}

// ---------------------------------------------------------------------------
// Per-row quantisation of a bf16 matrix to signed 8-bit integers (row_quant_s8).
// cols % 8 == 0.  T threads share a row and hold it in registers between the maximum
// and the rounding (NV 16-byte vectors each), so it is read once: bound by DRAM, 2
// bytes read and 1 written per element.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t bf16x8_abs_bits(const uint4& u) {   // largest magnitude of 8 bf16, as fp32 bits
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
  return m;
}
__device__ __forceinline__ uint2 bf16x8_to_s8(const uint4& u, const RowQuantS8& r) {
  float f[8];
  bf16x8_to_f32(u, f);
  return make_uint2(quant_s8x4(f[0], f[1], f[2], f[3], r), quant_s8x4(f[4], f[5], f[6], f[7], r));
}

template <int T, int NV>
__global__ void __launch_bounds__(T > 128 ? T : 128) quantize_rows_s8_kernel(const bf16* __restrict__ x, int rows, int cols,
                                                                            uint8_t* __restrict__ q,
                                                                            float* __restrict__ scale) {
  pdl_wait();
  pdl_trigger();
  constexpr int RPB = T > 128 ? 1 : 128 / T;       // rows per block
  const int t = threadIdx.x % T, nvec = cols / 8;
  const size_t row = static_cast<size_t>(blockIdx.x) * RPB + threadIdx.x / T;
  if (T < 128 && row >= static_cast<size_t>(rows)) return;   // whole warps; with T >= 128 a block is a row
  const uint4* xr = reinterpret_cast<const uint4*>(x + row * cols);
  uint4 v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = t + i * T < nvec ? xr[t + i * T] : make_uint4(0, 0, 0, 0);
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) amax = max(amax, bf16x8_abs_bits(v[i]));
  amax = warp_max_u32(amax);
  if (T > 32) {
    __shared__ uint32_t part[T / 32];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < T / 32; ++w) amax = max(amax, part[w]);
  }
  const RowQuantS8 r = row_quant_s8(amax);
  if (t == 0) scale[row] = r.scale;
  uint2* qr = reinterpret_cast<uint2*>(q + row * cols);
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (t + i * T < nvec) qr[t + i * T] = bf16x8_to_s8(v[i], r);
}

// rows longer than a block's registers hold: a block per row, read twice
__global__ void __launch_bounds__(256) quantize_long_rows_s8_kernel(const bf16* __restrict__ x, int cols,
                                                                    uint8_t* __restrict__ q, float* __restrict__ scale) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint32_t part[8];
  const size_t row = blockIdx.x;
  const uint4* xr = reinterpret_cast<const uint4*>(x + row * cols);
  uint2* qr = reinterpret_cast<uint2*>(q + row * cols);
  const int nvec = cols / 8;
  uint32_t amax = 0;
  for (int c = threadIdx.x; c < nvec; c += 256) amax = max(amax, bf16x8_abs_bits(xr[c]));
  amax = warp_max_u32(amax);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) amax = max(amax, part[w]);
  const RowQuantS8 r = row_quant_s8(amax);
  if (threadIdx.x == 0) scale[row] = r.scale;
  for (int c = threadIdx.x; c < nvec; c += 256) qr[c] = bf16x8_to_s8(xr[c], r);
}

// ---------------------------------------------------------------------------
// fp32 path: QK-RMSNorm (gain) then RoPE at the row's coordinates, in place on the
// q and k parts of qkv [rows, 3d].  One thread per (row, head, q|k).
// ---------------------------------------------------------------------------
struct RopeF32 {
  int dims[3];
  float th_hi[32];
  float th_lo[32];
};

__global__ void __launch_bounds__(128) qk_norm_rope_f32_kernel(float* __restrict__ qkv, int rows, int d, int heads,
                                                               const float* __restrict__ q_g,
                                                               const float* __restrict__ k_g, float eps,
                                                               const int4* __restrict__ pos, const RopeF32 rope) {
  const int hd = d / heads;
  const size_t idx = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (idx >= static_cast<size_t>(rows) * heads * 2) return;
  const int part = static_cast<int>(idx % 2);
  const int h = static_cast<int>((idx / 2) % heads);
  const size_t row = idx / (2 * heads);
  float* v = qkv + row * 3 * d + part * d + h * hd;
  const float* g = part ? k_g : q_g;
  float x[64];
  float ss = 0.f;
  for (int c = 0; c < hd; ++c) {
    x[c] = v[c];
    ss = fmaf(x[c], x[c], ss);
  }
  const float r = rsqrtf(ss / hd + eps);
  for (int c = 0; c < hd; ++c) x[c] = x[c] * r * g[c];
  const int4 p4 = pos[row];
  const float p[3] = {static_cast<float>(p4.x), static_cast<float>(p4.y), static_cast<float>(p4.z)};
  int off = 0, pair = 0;
  for (int a = 0; a < 3; ++a) {
    const int half = rope.dims[a] / 2;
    for (int j = 0; j < half; ++j) {
      float c, s;
      rope_cos_sin(p[a], rope.th_hi[pair + j], rope.th_lo[pair + j], c, s);
      const float xa = x[off + j], xb = x[off + j + half];
      x[off + j] = xa * c - xb * s;
      x[off + j + half] = xa * s + xb * c;
    }
    off += rope.dims[a];
    pair += half;
  }
  for (int c = 0; c < hd; ++c) v[c] = x[c];
}

// ---------------------------------------------------------------------------
// fp32 path: SIMT GEMM Y = A W^T (+ b) with the same epilogues as the tensor-core
// kernel (bias, GELU, residual, SwiGLU).  64 x 64 tiles, K slices of 16, 4 x 4 per
// thread.  EPI 3 (SwiGLU): N is the output width, W has 2N rows (gate rows, then
// up rows); a tile loads 32 gate rows and the 32 matching up rows, so that lane l
// (tx < 8) and lane l + 8 of a warp hold the gate and up sums of the same outputs.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float silu_f(float z) { return z / (1.0f + __expf(-z)); }

template <int EPI>
__global__ void __launch_bounds__(256) gemm_f32_kernel(const float* __restrict__ A, const float* __restrict__ W,
                                                       const float* __restrict__ bias, float* __restrict__ Y, int M,
                                                       int N, int K) {
  __shared__ float sA[16][64 + 4];
  __shared__ float sW[16][64 + 4];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int m0 = blockIdx.x * 64, n0 = blockIdx.y * (EPI == 3 ? 32 : 64);
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 16) {
    for (int i = threadIdx.x; i < 64 * 16; i += 256) {
      const int r = i / 16, c = i % 16;
      const int gm = m0 + r, gk = k0 + c;
      int gn = n0 + r;
      bool wok = gn < N;
      if (EPI == 3) {
        gn = n0 + (r & 31);
        wok = gn < N;
        gn += (r >> 5) * N;     // rows 32..63 of the tile: the up rows
      }
      sA[c][r] = (gm < M && gk < K) ? A[static_cast<size_t>(gm) * K + gk] : 0.f;
      sW[c][r] = (wok && gk < K) ? W[static_cast<size_t>(gn) * K + gk] : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 16; ++kk) {
      float a[4], w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = sA[kk][ty * 4 + i];
        w[i] = sW[kk][tx * 4 + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], w[j], acc[i][j]);
    }
    __syncthreads();
  }
  if (EPI == 3) {
    // lanes tx < 8 hold gate columns tx*4 + j, lanes tx + 8 the up columns
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float u = __shfl_down_sync(0xffffffffu, acc[i][j], 8);
        const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
        if (tx < 8 && m < M && n < N) {
          const float gv = acc[i][j] + (bias ? bias[n] : 0.f);
          const float uv = u + (bias ? bias[N + n] : 0.f);
          Y[static_cast<size_t>(m) * N + n] = silu_f(gv) * uv;
        }
      }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + ty * 4 + i;
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx * 4 + j;
      if (n >= N) continue;
      float v = acc[i][j] + (bias ? bias[n] : 0.f);
      float* y = Y + static_cast<size_t>(m) * N + n;
      if (EPI == 1) v = gelu_erf(v);
      if (EPI == 2) v += *y;
      *y = v;
    }
  }
}

}  // namespace ts
