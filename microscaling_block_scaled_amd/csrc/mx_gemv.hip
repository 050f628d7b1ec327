// mx_gemv.hip -- products of a few tokens with 4-bit MX weights for gfx950:
//   y[m, n] = sum over blocks b of 2^(s[n, b] - 127) * sum_{k in b} x[m, k] * P[n, k]
// with x in bf16, P in E2M1 and one E8M0 scale for 32 weights of a row.
//
// A weight times its scale is exact in bf16 (two significant bits times a power
// of two), so the products are exact and the sums run in fp32.
//
// Bound: HBM, 17 bytes for 32 weights that are each used once per token.  A
// workgroup owns 16 rows of W and all of K: its waves take K in steps of 512
// (4 KB of weights), their partial sums meet in LDS, and nothing is left to
// join across workgroups, so results do not depend on timing.  The weights are
// the 16-row operand of a 16x16x32 bf16 matrix instruction and the tokens its
// 16 columns: one token costs no more weight bytes or conversions than 16.  A
// lane (row l % 16, group g = l / 16) loads 16 bytes, the whole block 4 i + g of
// four, and feeds its elements 8 j .. 8 j + 7 to instruction j; the tokens' lanes
// take the same elements of x, which is all the order that a sum over k needs.
#include <cstdlib>
#include "mx_device.hpp"
#include "mx_layer.h"

namespace mx {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int ROWS = 16;    // rows of W per workgroup

// Eight E2M1 codes (a dword) times the scale as a bf16 operand.
__device__ __forceinline__ bf16x8 fp4_operand(uint32_t q, float scale) {
  union { bf16x2 p[4]; bf16x8 v; } u;
  u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0);
  u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1);
  u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2);
  u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3);
  return u.v;
}

// What a lane takes in one step of NI * 128 elements of K: block 4 i + g of its
// row of W at q[i], the block's scale at byte g of s[i], and the block's elements
// of its tokens at x[i][j][t].
template <int MT, int NI>
struct Step {
  uint4 q[NI];
  uint32_t s[NI];
  bf16x8 x[NI][4][MT];
};

// x[k .. k + 7] of a token, +0 past K; rows of x need no alignment beyond their
// type's.
template <bool WHOLE>
__device__ __forceinline__ bf16x8 load_x(const uint16_t* xrow, int64_t k, int64_t K) {
  union { uint16_t h[8]; bf16x8 v; uint4 u; } r;
  if (WHOLE || k + 8 <= K) {
    __builtin_memcpy(&r.u, xrow + k, 16);
  } else {
    r.u = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (k + e < K) r.h[e] = xrow[k + e];
  }
  return r.v;
}

// Blocks at or past nb read as zeros.
template <int MT, int NI, bool WHOLE>
__device__ __forceinline__ void load_step(Step<MT, NI>& st, const uint8_t* qrow, const uint8_t* srow,
                                          const uint16_t* const xrow[MT], int b0, int g, int nb, int64_t K) {
#pragma unroll
  for (int i = 0; i < NI; i++) {
    const int b = b0 + 4 * i + g;
    if (WHOLE || b < nb) st.q[i] = *(const uint4*)(qrow + (int64_t)b * 16);
    else st.q[i] = make_uint4(0, 0, 0, 0);
  }
  if (WHOLE) {
    __builtin_memcpy(st.s, srow + b0, 4 * NI);  // any alignment: rows of scales are nb bytes
  } else {
#pragma unroll
    for (int i = 0; i < NI; i++) {
      const int b = b0 + 4 * i + g;
      st.s[i] = b < nb ? (uint32_t)srow[b] << (8 * g) : 0u;
    }
  }
#pragma unroll
  for (int i = 0; i < NI; i++)
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int t = 0; t < MT; t++)
        st.x[i][j][t] = load_x<WHOLE>(xrow[t], (int64_t)(b0 + 4 * i + g) * 32 + 8 * j, K);
}

template <int MT, int NI>
__device__ __forceinline__ void take_step(const Step<MT, NI>& st, int g, f32x4 acc[MT]) {
#pragma unroll
  for (int i = 0; i < NI; i++) {
    const uint32_t code = (st.s[i] >> (8 * g)) & 0xFFu;
    const float scale = __builtin_bit_cast(float, code << 23);
    const uint32_t w[4] = {st.q[i].x, st.q[i].y, st.q[i].z, st.q[i].w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const bf16x8 a = fp4_operand(w[j], scale);
#pragma unroll
      for (int t = 0; t < MT; t++)
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, st.x[i][j][t], acc[t], 0, 0, 0);
    }
  }
}

template <int MT, int NI, int WAVES, int OCC, bool BF16>
__global__ __launch_bounds__(64 * WAVES, OCC) void k_gemv(GemvArgs p) {
  __shared__ float part[WAVES][MT][16][ROWS + 1];
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * ROWS, m0 = (int64_t)blockIdx.y * (16 * MT);
  const int nb = (int)((p.K + 31) >> 5);
  // rows past N read row N - 1 again and are not stored
  const int64_t n = n0 + (lane & 15) < p.N ? n0 + (lane & 15) : p.N - 1;
  const uint8_t* qrow = p.wq + n * nb * 16;
  const uint8_t* srow = p.ws + n * nb;
  const uint16_t* xrow[MT];
  f32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; t++) {  // tokens past M read the first token's row and are not stored
    const int64_t m = m0 + 16 * t + (lane & 15);
    xrow[t] = p.x + (m < p.M ? m : m0) * p.ld_x;
    acc[t] = f32x4{0, 0, 0, 0};
  }
  constexpr int STEP = 4 * NI;                 // blocks a wave takes at a time
  const int whole = (int)(p.K / (32 * STEP));  // steps with all of their blocks and elements
  int s = wave;
  for (; s < whole; s += WAVES) {
    Step<MT, NI> st;
    load_step<MT, NI, true>(st, qrow, srow, xrow, s * STEP, g, nb, p.K);
    take_step<MT, NI>(st, g, acc);
  }
  if (s == whole && whole * STEP < nb) {  // the short last step
    Step<MT, NI> st;
    load_step<MT, NI, false>(st, qrow, srow, xrow, s * STEP, g, nb, p.K);
    take_step<MT, NI>(st, g, acc);
  }
  // lane (g, m) holds rows 4 g .. 4 g + 3 of token m
#pragma unroll
  for (int t = 0; t < MT; t++)
#pragma unroll
    for (int r = 0; r < 4; r++) part[wave][t][lane & 15][4 * g + r] = acc[t][r];
  __syncthreads();
  for (int i = threadIdx.x; i < 256 * MT; i += 64 * WAVES) {
    const int t = i >> 8, m = (i >> 4) & 15, r = i & 15;
    if (m0 + 16 * t + m >= p.M || n0 + r >= p.N) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; w++) v += part[w][t][m][r];
    const int64_t at = (m0 + 16 * t + m) * p.ld_y + n0 + r;
    if (BF16) ((uint16_t*)p.y)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
    else ((float*)p.y)[at] = v;
  }
}

}  // namespace

template <int MT, int NI, int W, int OCC>
static void go(const GemvArgs& a, dim3 g, hipStream_t st) {
  if (a.bf16) hipLaunchKernelGGL((k_gemv<MT, NI, W, OCC, true>), g, dim3(64 * W), 0, st, a);
  else hipLaunchKernelGGL((k_gemv<MT, NI, W, OCC, false>), g, dim3(64 * W), 0, st, a);
}
hipError_t launch_gemv(const GemvArgs& a, hipStream_t st) {
  const unsigned gx = (unsigned)((a.N + ROWS - 1) / ROWS);
  static const int V = getenv("MXV") ? atoi(getenv("MXV")) : 0;
  if (a.M <= 16) {
    const dim3 g(gx, 1);
    switch (V) {
      case 0: go<1, 4, 8, 4>(a, g, st); break;
      case 1: go<1, 2, 8, 4>(a, g, st); break;
      case 2: go<1, 2, 8, 8>(a, g, st); break;
      case 3: go<1, 4, 16, 4>(a, g, st); break;
      case 4: go<1, 2, 16, 8>(a, g, st); break;
      case 5: go<1, 2, 16, 4>(a, g, st); break;
      case 6: go<1, 4, 4, 4>(a, g, st); break;
      case 7: go<1, 2, 4, 8>(a, g, st); break;
    }
  } else {  // each 32 tokens read the weights once
    const dim3 g(gx, (unsigned)((a.M + 31) / 32));
    go<2, 2, 8, 4>(a, g, st);
  }
  return hipGetLastError();
}

}  // namespace mx
