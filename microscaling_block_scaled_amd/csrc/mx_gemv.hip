// mx_gemv.hip -- products of a few tokens with 4-bit MX weights for gfx950:
//   y[m, n] = sum over blocks b of 2^(s[n, b] - 127) * sum_{k in b} x[m, k] * P[n, k]
// with x in bf16, P in E2M1 and one E8M0 scale for 32 weights of a row.
//
// A weight times its scale is exact in bf16 (two significant bits times a power
// of two), so the products are exact and the sums run in fp32.
//
// Bound: HBM, 17 bytes for 32 weights that are each used once per token; for 16
// tokens and more also the reading of x by each workgroup.  A workgroup owns 16 R
// rows of W and all of K: its waves take a run of K each, in steps of 128 NI
// elements, their partial sums meet in LDS, and nothing is left to join across
// workgroups, so results do not depend on timing.  The weights are the 16-row
// operand of a 16x16x32 bf16 matrix instruction and the tokens its 16 columns: one
// token costs no more weight bytes or conversions than 16.  A lane (row l % 16,
// group g = l / 16) takes the whole block 4 i + g of four and feeds its elements
// 8 j .. 8 j + 7 to instruction j; the tokens' lanes take the same elements of x,
// which is all the order that a sum over k needs.
//
// Weights and x go through LDS, each wave's own piece, without a barrier: neighbouring
// lanes then load neighbouring pieces of a row.  With each lane loading its own row of
// the operand, 4 x 14336 x 4096 took 12.4 us instead of 8.1 (31 MB: 3.9 TB/s),
// 16 x 4096 x 14336 19.3 instead of 11.6 (32 MB, and 117 MB of x out of the L2s: the
// loads of a CU take 10000 of its 25000 cycles, its LDS as many).
#include "mx_device.hpp"
#include "mx_layer.h"

namespace mx {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Eight E2M1 codes (a dword) times the scale as a bf16 operand.
__device__ __forceinline__ bf16x8 fp4_operand(uint32_t q, float scale) {
  union { bf16x2 p[4]; bf16x8 v; } u;
  u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0);
  u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1);
  u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2);
  u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3);
  return u.v;
}

// One wave's piece of LDS, which holds a step of 128 NI elements of K.  All loads take
// whole runs of a row, 64 NI bytes of weights and 256 NI of x.
template <int TOK, int NI, int R>
struct Step {
  static constexpr int ROWS = 16 * R;
  static constexpr int Q_PITCH = 64 * NI + 16, X_PITCH = 256 * NI + 16, S_PITCH = 64 + 16;  // other banks for each row
  static constexpr int Q_AT = 0, S_AT = Q_AT + ROWS * Q_PITCH, X_AT = S_AT + ROWS * S_PITCH;
  static constexpr int BYTES = X_AT + TOK * X_PITCH;
  static constexpr int XL = (TOK * NI + 3) / 4;
  static constexpr int SCALED = 64 / (4 * NI);  // steps that one load of scales serves
};

struct Rows {
  const uint8_t* q;  // first row of the workgroup
  const uint8_t* s;
  const uint16_t* x;  // first token
  int64_t ld_x, K;
  int nb, rows, live;  // rows and tokens that there are
};

// Rows and tokens past the last are the last.  Blocks at or past `end`, and pieces of x
// that are not whole within K, take the first weights' bytes in their place: every
// step then has the same number of loads, which is what lets a wait leave the later
// steps' loads in flight.
template <int TOK, int NI, int R>
__device__ __forceinline__ void load_weights(u32x4 (&q)[R * NI], const Rows& w, int b0, int end) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < R * NI; r++) {
    const int f = 64 * r + lane, row = f / (4 * NI), b = b0 + f % (4 * NI);
    const int64_t at = ((int64_t)(row < w.rows ? row : w.rows - 1) * w.nb + b) * 16;
    q[r] = *(const u32x4*)(w.q + (b < end ? at : 0));
  }
}
template <int TOK, int NI, int R, int XL>
__device__ __forceinline__ void load_tokens(u32x4 (&x)[XL], const Rows& w, int b0, int end) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < XL; r++) {
    const int f = 64 * r + lane, tok = f / (16 * NI);
    const int64_t k = (int64_t)b0 * 32 + 8 * (f % (16 * NI));
    const uint8_t* src = (const uint8_t*)(w.x + (tok < w.live ? tok : w.live - 1) * w.ld_x + k);
    __builtin_memcpy(&x[r], b0 < end && k + 8 <= w.K ? src : w.q, 16);
  }
}
// what load_tokens left out of a step that K ends in: the last elements, and zeros
template <int TOK, int NI, int R, int XL>
__device__ __forceinline__ void mend_tokens(u32x4 (&x)[XL], const Rows& w, int b0) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < XL; r++) {
    const int f = 64 * r + lane, tok = f / (16 * NI);
    const int64_t k = (int64_t)b0 * 32 + 8 * (f % (16 * NI));
    if (k + 8 <= w.K) continue;
    const uint16_t* src = w.x + (tok < w.live ? tok : w.live - 1) * w.ld_x + k;
    uint32_t h[8] = {};
    if (k < w.K) {
#pragma unroll
      for (int e = 0; e < 8; e++) h[e] = src[k + e < w.K ? e : 0];
    }
#pragma unroll
    for (int e = 0; e < 8; e++) h[e] = k + e < w.K ? h[e] : 0;
#pragma unroll
    for (int i = 0; i < 4; i++) x[r][i] = h[2 * i] | h[2 * i + 1] << 16;
  }
}
// Scales of the 64 blocks from b0 on, 16 blocks to each of four lanes a row.  Runs that
// a row ends in are left to mend_scales.
template <int R>
__device__ __forceinline__ void load_scales(u32x4 (&s)[R], const Rows& w, int b0) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int a = 0; a < R; a++) {
    const int row = 16 * a + lane / 4, b = b0 + 16 * (lane & 3);
    const uint8_t* src = w.s + (int64_t)(row < w.rows ? row : w.rows - 1) * w.nb + b;
    __builtin_memcpy(&s[a], b + 16 <= w.nb ? src : w.q, 16);  // any alignment: rows of scales are nb bytes
  }
}
template <int R>
__device__ __forceinline__ void mend_scales(u32x4 (&s)[R], const Rows& w, int b0, int end) {
  const int lane = threadIdx.x & 63, b = b0 + 16 * (lane & 3);
  if (b >= end || b + 16 <= w.nb) return;  // runs past `end` are of no step
#pragma unroll
  for (int a = 0; a < R; a++) {
    const int row = 16 * a + lane / 4;
    const uint8_t* src = w.s + (int64_t)(row < w.rows ? row : w.rows - 1) * w.nb + b;
    uint32_t c[16];
#pragma unroll
    for (int e = 0; e < 16; e++) c[e] = src[b + e < w.nb ? e : 0];
#pragma unroll
    for (int e = 0; e < 16; e++) c[e] = b + e < w.nb ? c[e] : 0;
#pragma unroll
    for (int i = 0; i < 4; i++) s[a][i] = c[4 * i] | c[4 * i + 1] << 8 | c[4 * i + 2] << 16 | c[4 * i + 3] << 24;
  }
}
template <int TOK, int NI, int R>
__device__ __forceinline__ void stage_weights(const u32x4 (&q)[R * NI], uint8_t* lds) {
  using St = Step<TOK, NI, R>;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < R * NI; r++) {
    const int f = 64 * r + lane;
    *(u32x4*)(lds + St::Q_AT + f / (4 * NI) * St::Q_PITCH + f % (4 * NI) * 16) = q[r];
  }
}
template <int TOK, int NI, int R, int XL>
__device__ __forceinline__ void stage_tokens(const u32x4 (&x)[XL], uint8_t* lds) {
  using St = Step<TOK, NI, R>;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < XL; r++) {
    const int f = 64 * r + lane;
    if (TOK * NI < 4 && f >= 16 * NI * TOK) break;  // fewer lanes hold a piece
    *(u32x4*)(lds + St::X_AT + f / (16 * NI) * St::X_PITCH + f % (16 * NI) * 16) = x[r];
  }
}
template <int TOK, int NI, int R>
__device__ __forceinline__ void stage_scales(const u32x4 (&s)[R], uint8_t* lds) {
  using St = Step<TOK, NI, R>;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int a = 0; a < R; a++) *(u32x4*)(lds + St::S_AT + (16 * a + lane / 4) * St::S_PITCH + 16 * (lane & 3)) = s[a];
}
// lanes of one wave: what one wrote to LDS, the others read
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Step `at` of those that the staged scales serve.
template <int TOK, int NI, int R>
__device__ __forceinline__ void take_step(const uint8_t* lds, int at, f32x4 (&acc)[R][(TOK + 15) / 16]) {
  using St = Step<TOK, NI, R>;
  constexpr int MT = (TOK + 15) / 16;
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
#pragma unroll
  for (int i = 0; i < NI; i++) {
    uint4 q[R];
    float scale[R];
#pragma unroll
    for (int a = 0; a < R; a++) {
      q[a] = *(const uint4*)(lds + St::Q_AT + (16 * a + m) * St::Q_PITCH + (4 * i + g) * 16);
      const uint32_t code = lds[St::S_AT + (16 * a + m) * St::S_PITCH + 4 * NI * at + 4 * i + g];
      scale[a] = __builtin_bit_cast(float, code << 23);
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
      bf16x8 b[MT];
#pragma unroll
      for (int t = 0; t < MT; t++) {
        const int tok = (16 * t + m) & (TOK - 1);  // columns past TOK repeat the first ones
        b[t] = *(const bf16x8*)(lds + St::X_AT + tok * St::X_PITCH + (4 * i + g) * 64 + 16 * j);
      }
#pragma unroll
      for (int a = 0; a < R; a++) {
        const bf16x8 w = fp4_operand(j == 0 ? q[a].x : j == 1 ? q[a].y : j == 2 ? q[a].z : q[a].w, scale[a]);
#pragma unroll
        for (int t = 0; t < MT; t++)
          acc[a][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, b[t], acc[a][t], 0, 0, 0);
      }
    }
  }
}

// TOK tokens (1, 2, 4, 8, 16 or 32) and 16 R rows of W by one workgroup; weights D
// steps ahead.
template <int TOK, int NI, int WAVES, int R, int D, bool BF16>
__global__ __launch_bounds__(64 * WAVES) void k_gemv(GemvArgs p) {
  using St = Step<TOK, NI, R>;
  constexpr int MT = (TOK + 15) / 16, ROWS = 16 * R, XL = St::XL;
  constexpr int PART = 4 * MT * 16 * (ROWS + 1);  // bytes of a wave's partial sums
  __shared__ __align__(16) uint8_t lds[WAVES * (St::BYTES > PART ? St::BYTES : PART)];
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * ROWS, m0 = (int64_t)blockIdx.y * TOK;
  Rows w;
  w.nb = (int)((p.K + 31) >> 5);
  w.K = p.K;
  w.q = p.wq + n0 * w.nb * 16;
  w.s = p.ws + n0 * w.nb;
  w.x = p.x + m0 * p.ld_x;
  w.ld_x = p.ld_x;
  w.rows = p.N - n0 < ROWS ? (int)(p.N - n0) : ROWS;
  w.live = p.M - m0 < TOK ? (int)(p.M - m0) : TOK;
  const int live = w.live;
  f32x4 acc[R][MT];
#pragma unroll
  for (int a = 0; a < R; a++)
#pragma unroll
    for (int t = 0; t < MT; t++) acc[a][t] = f32x4{0, 0, 0, 0};
  uint8_t* mine = lds + wave * St::BYTES;
  constexpr int STEP = 4 * NI;  // blocks a wave takes at a time
  const int steps = (w.nb + STEP - 1) / STEP, per = (steps + WAVES - 1) / WAVES;
  int s = wave * per;
  const int end = s + per < steps ? s + per : steps;
  if (s < end) {
    const int last = end * STEP < w.nb ? end * STEP : w.nb;
    u32x4 q[D][R * NI], x[XL], sc[R];
    load_scales(sc, w, s * STEP);
#pragma unroll
    for (int d = 0; d < D; d++) {
      if (d == 0) load_tokens<TOK, NI, R>(x, w, s * STEP, last);
      load_weights<TOK, NI, R>(q[d], w, (s + d) * STEP, last);
    }
    mend_scales(sc, w, s * STEP, last);
    stage_scales<TOK, NI, R>(sc, mine);
    // one exit, at the end of D steps: with one at each, a wait would have to cover
    // the loads of whichever step came last
    for (int at = 0; s < end;) {
      const bool turn = at == St::SCALED - D;  // the D steps after these need other scales
      if (turn) load_scales(sc, w, s + D < end ? (s + D) * STEP : w.nb);
#pragma unroll
      for (int d = 0; d < D; d++) {
        const bool live = d == 0 || s < end;
        if (live) {
          if ((int64_t)(s + 1) * STEP * 32 > p.K) mend_tokens<TOK, NI, R>(x, w, s * STEP);
          stage_weights<TOK, NI, R>(q[d], mine);
          stage_tokens<TOK, NI, R>(x, mine);
          wave_fence();
        }
        load_tokens<TOK, NI, R>(x, w, (s + 1) * STEP, last);
        load_weights<TOK, NI, R>(q[d], w, (s + D) * STEP, last);
        if (live) {
          take_step<TOK, NI, R>(mine, at + d, acc);
          wave_fence();
        }
        s++;
      }
      at += D;
      if (turn) {
        mend_scales(sc, w, s * STEP, last);
        stage_scales<TOK, NI, R>(sc, mine);
        at = 0;
      }
    }
  }
  __syncthreads();
  // lane (g, m) holds rows 4 g .. 4 g + 3 of token m
  float* part = (float*)lds;
  auto at = [](int w, int m, int r) { return (w * MT * 16 + m) * (ROWS + 1) + r; };
#pragma unroll
  for (int a = 0; a < R; a++)
#pragma unroll
    for (int t = 0; t < MT; t++)
#pragma unroll
      for (int r = 0; r < 4; r++) part[at(wave, 16 * t + (lane & 15), 16 * a + 4 * g + r)] = acc[a][t][r];
  __syncthreads();
  for (int i = threadIdx.x; i < TOK * ROWS; i += 64 * WAVES) {
    const int m = i / ROWS, r = i % ROWS;
    if (m >= live || n0 + r >= p.N) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; w++) v += part[at(w, m, r)];
    const int64_t to = (m0 + m) * p.ld_y + n0 + r;
    if (BF16) ((uint16_t*)p.y)[to] = __builtin_bit_cast(uint16_t, (__bf16)v);
    else ((float*)p.y)[to] = v;
  }
}

template <int TOK, int NI, int WAVES, int R, int D>
void go(const GemvArgs& a, hipStream_t st) {
  const dim3 g((unsigned)((a.N + 16 * R - 1) / (16 * R)), (unsigned)((a.M + TOK - 1) / TOK)), b(64 * WAVES);
  if (a.bf16) hipLaunchKernelGGL((k_gemv<TOK, NI, WAVES, R, D, true>), g, b, 0, st, a);
  else hipLaunchKernelGGL((k_gemv<TOK, NI, WAVES, R, D, false>), g, b, 0, st, a);
}

}  // namespace

// Where 16-row groups are fewer than two for each of the 256 CUs, eight waves share
// a group's K; where there are more, four do, so that more workgroups fit on a CU,
// and for many tokens a workgroup takes several groups, since each group reads all
// of x.  Measured (us, eight waves and one group / the other form):
//   1 x 4096 x 14336   7.9 / 10.6     1 x 14336 x 4096    8.1 / 7.7
//   4 x 14336 x 4096   9.2 / 8.3      16 x 14336 x 4096  17.9 / 11.1 (two groups)
//   16 x 4096 x 14336 11.9 / 19.3     32 x 14336 x 14336 71.0 / 45.0 (four groups)
// Weights are loaded one step ahead, for 32 tokens, whose steps are half as wide, two
// (one / two steps ahead, us): 32 x 4096 x 4096 7.6 / 7.3, 32 x 14336 x 14336 41.2 / 36.0,
// but 4 x 14336 x 4096 8.1 / 9.1, 1 x 4096 x 14336 7.9 / 8.5, 16 x 4096 x 14336 11.9 / 12.4.
hipError_t launch_gemv(const GemvArgs& a, hipStream_t st) {
  const bool many = (a.N + 15) / 16 > 512;
  if (a.M == 1) many ? go<1, 2, 4, 1, 1>(a, st) : go<1, 2, 8, 1, 1>(a, st);
  else if (a.M == 2) many ? go<2, 2, 4, 1, 1>(a, st) : go<2, 2, 8, 1, 1>(a, st);
  else if (a.M <= 4) many ? go<4, 2, 4, 1, 1>(a, st) : go<4, 2, 8, 1, 1>(a, st);
  else if (a.M <= 8) many ? go<8, 2, 4, 1, 1>(a, st) : go<8, 2, 8, 1, 1>(a, st);
  else if (a.M <= 16) many ? go<16, 2, 4, 2, 1>(a, st) : go<16, 2, 8, 1, 1>(a, st);
  else many ? go<32, 1, 4, 4, 2>(a, st) : go<32, 1, 8, 1, 2>(a, st);  // 32 tokens a reading of the weights
  return hipGetLastError();
}

}  // namespace mx
