// mx_attention.hip -- the paged 8-bit MX key/value cache and attention over it,
// for gfx950.
//
// Cache: pages of `page` tokens; elements [pages][heads][page][dim] in E4M3 or
// E5M2, scales [pages][heads][page][dim / 32].  A block of 32 consecutive values
// of one token's head shares an E8M0 scale (Algorithm 1 of "Microscaling Data
// Formats for Deep Learning", summary section 3, round to nearest even), so a
// token is appended without touching another one.
//
// Attention, for query token i of Lq and the tokens t < len - Lq + i + 1:
//   s_t = scale * q . k_t     p_t = exp(s_t - max s)     l = sum p_t
//   o = sum p_t v_t / l       lse = max s + log(l)
#include "mx_layer.h"
#include "mx_rows.hpp"
#include "mx_wave.hpp"

namespace mx {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// cache write
// ---------------------------------------------------------------------------
// A lane takes 8 elements of a token's head, a quad one block.  Bound: HBM.
template <int SRC, int F>
__global__ __launch_bounds__(256) void k_cache_write(CacheWriteArgs p) {
  constexpr int ESZ = SRC == SRC_BF16 ? 2 : 4;
  const int chunks = p.c.dim / 8, per = 2 * p.c.heads * chunks;  // of a token: keys, then values
  const int64_t n = p.tokens * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t tok = i / per;
    int rest = (int)(i - tok * per);
    const bool value = rest >= per / 2;
    if (value) rest -= per / 2;
    const int head = rest / chunks, c = rest - head * chunks;
    const int64_t slot = p.slots[tok];  // the same for the lanes of a quad
    if (slot < 0 || slot >= p.c.pages * p.c.page) continue;
    const uint8_t* src = value ? (const uint8_t*)p.v + tok * p.ld_v + head * p.hs_v
                               : (const uint8_t*)p.k + tok * p.ld_k + head * p.hs_k;
    uint32_t raw[2 * ESZ], v[8], am = 0, rnd[8];
    load_elems<ESZ, 8, false>(src + (int64_t)c * 8 * ESZ, 8, raw);
    widen8<SRC>(raw, v);
#pragma unroll
    for (int k = 0; k < 8; k++) am = umax(am, v[k] & 0x7FFFFFFFu);
    am = umax(am, quad_xor1(am));
    am = umax(am, quad_xor2(am));
    const uint32_t code = scale_code<F>(am);
    const int64_t pg = slot / p.c.page;
    const int64_t row = (pg * p.c.heads + head) * p.c.page + (slot - pg * p.c.page);
    if ((c & 3) == 0) (value ? p.c.v_s : p.c.k_s)[row * (p.c.dim / 32) + (c >> 2)] = (uint8_t)code;
    store8<F, false>((value ? p.c.v_q : p.c.k_q) + row * p.c.dim, c, convert8<F, false>(v, code, rnd));
  }
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
// Rows of a key/value head are its (query token, query head) pairs; a workgroup
// takes NR tiles of 16 of them and one piece of the request's tokens, its four
// waves 32 tokens at a time.  Both products run on 16x16x32 bf16 matrix
// instructions, to which an element times its scale is exact, straight from
// registers:
//   S^T = K Q^T   lane (l % 16, g = l / 16) loads dims g D/4 .. of token l % 16
//                 and feeds dims 8 j .. of them to instruction j, as the lane of
//                 Q does; it gets rows' scores of tokens 4 g .. 4 g + 3
//   O^T = V^T P^T those 8 scores (two groups of 16 tokens) are the lane's 8 of
//                 the 32 of a sum over tokens as they are; the lane loads dims
//                 (l % 16) D/16 .. of the same 8 tokens and transposes 2 x 2
// so neither P nor V passes through LDS.  P is rounded to bf16 (relative error
// 2^-9, of the size of the output's own rounding); scores, maxima, sums and O
// stay in fp32.
constexpr int WAVES = 4;
constexpr int STEP = 32;  // tokens a wave takes at a time

struct AttnArgs {
  AttentionArgs a;
  int rows;              // Lq * group
  int splits;
  int chunk;             // tokens of a piece, a multiple of STEP * WAVES
  uint32_t page16, magic;  // page / 16 and the constant that divides by it
  float* part_o;         // [B][heads][rows][splits][dim]
  float* part_ml;        // [B][heads][rows][splits][2]
};

template <int F>
__device__ __forceinline__ uint32_t cvt_lo(uint32_t w, float s) {
  bf16x2 r;
  if constexpr (F == E4M3) r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false);
  else r = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, s, false);
  return __builtin_bit_cast(uint32_t, r);
}
template <int F>
__device__ __forceinline__ uint32_t cvt_hi(uint32_t w, float s) {
  bf16x2 r;
  if constexpr (F == E4M3) r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true);
  else r = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, s, true);
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ float e8m0(uint32_t code) { return __builtin_bit_cast(float, code << 23); }

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {  // N dwords, aligned to their size
  if constexpr (N == 1) {
    w[0] = *(const uint32_t*)p;
  } else if constexpr (N == 2) {
    const uint2 t = *(const uint2*)p;
    w[0] = t.x; w[1] = t.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; i++) {
      const uint4 t = *(const uint4*)(p + 16 * i);
      w[4 * i] = t.x; w[4 * i + 1] = t.y; w[4 * i + 2] = t.z; w[4 * i + 3] = t.w;
    }
  }
}

// The bytes of 32 tokens in a lane.
template <int D>
struct Raw {
  uint32_t k[2][D / 16];     // dims g D/4 .. of token 16 u + l % 16
  uint32_t ks[2];            // the scales of those dims (one, or two for 256)
  uint32_t v[2][4][D / 64];  // dims (l % 16) D/16 .. of token 16 u + 4 g + r
  uint32_t vs[2][D / 32];    // the scales of tokens 16 u + 4 g .. + 3, D / 32 bytes each
};

// Where tokens 16 u .. of a request lie: row (page, head, place) of the cache.
// A page that is not one of the cache's holds no tokens.
__device__ __forceinline__ bool locate(const AttnArgs& p, const int32_t* table, int head, int tok, int64_t& row) {
  const uint32_t i16 = (uint32_t)tok >> 4;
  const uint32_t idx = p.page16 == 1 ? i16 : __umulhi(i16, p.magic);
  const int pg = table[idx];
  row = ((int64_t)pg * p.a.c.heads + head) * p.a.c.page + (int)(i16 - idx * p.page16) * 16;
  return (uint32_t)pg < (uint32_t)p.a.c.pages;
}

// Rows are the same for the whole wave, so addresses are a scalar base and a
// lane's constant offset.
template <int D>
__device__ __forceinline__ uint32_t load_step(const AttnArgs& p, const int32_t* table, int head, int t0, int end,
                                              Raw<D>& x) {
  const uint32_t lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  uint32_t there = 0;
#pragma unroll
  for (int u = 0; u < 2; u++) {
    int64_t row = 0;
    bool ok = t0 + 16 * u < end;
    if (ok) ok = locate(p, table, head, t0 + 16 * u, row);
    if (!ok) row = 0;  // any row of the cache: what it holds is masked
    there |= (uint32_t)ok << u;
    const uint8_t* kq = p.a.c.k_q + row * D;
    const uint8_t* ks = p.a.c.k_s + row * (D / 32);
    const uint8_t* vq = p.a.c.v_q + row * D;
    const uint8_t* vs = p.a.c.v_s + row * (D / 32);
    load_words<D / 16>(kq + (i * D + g * (D / 4)), x.k[u]);
    if constexpr (D == 256) x.ks[u] = *(const uint16_t*)(ks + (i * 8 + 2 * g));
    else x.ks[u] = ks[i * (D / 32) + g * D / 128];
#pragma unroll
    for (int r = 0; r < 4; r++) load_words<D / 64>(vq + (4 * g * D + i * (D / 16)) + r * D, x.v[u][r]);
    load_words<D / 32>(vs + 4 * g * (D / 32), x.vs[u]);
  }
  return there;
}

__device__ __forceinline__ bf16x8 operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8, make_uint4(a, b, c, d));
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// Scale code of the lane's dims of V for token 16 u + 4 g + r: byte r D/32 +
// block of x.vs[u].
template <int D>
__device__ __forceinline__ uint32_t v_scale(const Raw<D>& x, int u, int r) {
  const int blk = (int)(threadIdx.x & 15) * (D / 16) / 32;
  if constexpr (D == 64) return (x.vs[u][r >> 1] >> (16 * (r & 1) + 8 * blk)) & 0xFFu;
  else if constexpr (D == 128) return (x.vs[u][r] >> (8 * blk)) & 0xFFu;
  else return ((blk & 4 ? x.vs[u][2 * r + 1] : x.vs[u][2 * r]) >> (8 * (blk & 3))) & 0xFFu;
}

// V as operands of the second product: dims (l % 16) D/16 + 4 k .. + 3 of the
// lane's 8 tokens (dword c of an operand: tokens 2 c and 2 c + 1 of the eight).
template <int D, int F>
__device__ __forceinline__ void v_operands(const Raw<D>& x, const float s[2][4], int k, uint32_t w[4][4]) {
#pragma unroll
  for (int u = 0; u < 2; u++)
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const uint32_t ra = x.v[u][2 * h][k], rb = x.v[u][2 * h + 1][k];
      const uint32_t a0 = cvt_lo<F>(ra, s[u][2 * h]), a1 = cvt_hi<F>(ra, s[u][2 * h]);
      const uint32_t b0 = cvt_lo<F>(rb, s[u][2 * h + 1]), b1 = cvt_hi<F>(rb, s[u][2 * h + 1]);
      w[0][2 * u + h] = __builtin_amdgcn_perm(b0, a0, 0x05040100u);
      w[1][2 * u + h] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
      w[2][2 * u + h] = __builtin_amdgcn_perm(b1, a1, 0x05040100u);
      w[3][2 * u + h] = __builtin_amdgcn_perm(b1, a1, 0x07060302u);
    }
}

// What a wave has summed for its rows.
template <int D, int NR>
struct Sums {
  f32x4 o[NR][D / 16];  // dim (4 g + e) D/16 + d of row l % 16
  float m[NR], l[NR];   // l over the lane's tokens only
};

// One step of 32 tokens.  `cut`: some row does not see all of them, or some are
// not there.  limit[n] is the number of them that the lane's row sees (less than
// 1: none, 32 or more: all), `end` the largest such number of the workgroup.
template <int D, int F, int NR>
__device__ __forceinline__ void take_step(const AttnArgs& p, Raw<D>& x, const bf16x8 (&q)[NR][D / 32],
                                          float scale2, bool cut, uint32_t there, int end,
                                          const int (&limit)[NR], Sums<D, NR>& sum) {
  const int g = (threadIdx.x & 63) >> 4;
  f32x4 s[NR][2];
#pragma unroll
  for (int u = 0; u < 2; u++) {
#pragma unroll
    for (int n = 0; n < NR; n++) s[n][u] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < D / 32; j++) {
      const uint32_t code = D == 256 ? (x.ks[u] >> (8 * (j >> 2))) & 0xFFu : x.ks[u];
      const float ks = e8m0(code);
      const uint32_t w0 = x.k[u][2 * j], w1 = x.k[u][2 * j + 1];
      const bf16x8 k = operand(cvt_lo<F>(w0, ks), cvt_hi<F>(w0, ks), cvt_lo<F>(w1, ks), cvt_hi<F>(w1, ks));
#pragma unroll
      for (int n = 0; n < NR; n++) s[n][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[n][j], s[n][u], 0, 0, 0);
    }
  }
  bool odd = false;
  if (cut) {
#pragma unroll
    for (int n = 0; n < NR; n++)
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const int tok = 16 * (e >> 2) + 4 * g + (e & 3);
        const bool seen = tok < limit[n] && (there >> (e >> 2) & 1);
        s[n][e >> 2][e & 3] = seen ? s[n][e >> 2][e & 3] : -__builtin_inff();
      }
    // Tokens that no row sees count as zeros whatever the cache holds there, for
    // 0 * NaN is not 0.  Of the others, one with a value that may not be finite
    // sends the step the long way (below) where rows see different tokens.
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
      for (int r = 0; r < 4; r++) {
        const bool gone = !(there >> u & 1) || 16 * u + 4 * g + r >= end;
        odd |= !gone && v_scale<D>(x, u, r) > (uint32_t)(254 - Fmt<F>::emax);
#pragma unroll
        for (int k = 0; k < D / 64; k++) {
          x.v[u][r][k] = gone ? 0u : x.v[u][r][k];
          odd |= (((x.v[u][r][k] & 0x7F7F7F7Fu) + (F == E4M3 ? 0x01010101u : 0x04040404u)) & 0x80808080u) != 0;
        }
      }
  }
  float vs[2][4];
#pragma unroll
  for (int u = 0; u < 2; u++)
#pragma unroll
    for (int r = 0; r < 4; r++) vs[u][r] = e8m0(v_scale<D>(x, u, r));
  if (cut) {  // a scale of a token that is not there may be a NaN
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
      for (int r = 0; r < 4; r++)
        vs[u][r] = !(there >> u & 1) || 16 * u + 4 * g + r >= end ? 1.0f : vs[u][r];
  }
  bf16x8 pr[NR];
#pragma unroll
  for (int n = 0; n < NR; n++) {
    float v[8], top = -__builtin_inff();
#pragma unroll
    for (int e = 0; e < 8; e++) {
      v[e] = s[n][e >> 2][e & 3] * scale2;
      top = __builtin_fmaxf(top, v[e]);
    }
    const float m = __builtin_fmaxf(sum.m[n], rows_max(top));
    const float base = m == -__builtin_inff() ? 0.0f : m;  // nothing seen yet: every p is 0
    if (__any(m != sum.m[n])) {
      const float a = __builtin_amdgcn_exp2f(sum.m[n] - base);
      sum.m[n] = m;
      sum.l[n] *= a;
#pragma unroll
      for (int d = 0; d < D / 16; d++) sum.o[n][d] *= a;
    }
#pragma unroll
    for (int e = 0; e < 8; e++) {
      v[e] = __builtin_amdgcn_exp2f(v[e] - base);
      sum.l[n] += v[e];
    }
    pr[n] = operand(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
  }
  if (p.a.Lq > 1 && __any(odd)) {
    // each number of tokens by itself, with the values past it cut, for the rows
    // that see that many
    for (int lim = 1; lim <= STEP; lim++) {
      uint32_t keep[4];
#pragma unroll
      for (int c = 0; c < 4; c++) {
        const int tok = 16 * (c >> 1) + 4 * g + 2 * (c & 1);
        keep[c] = (tok < lim ? 0xFFFFu : 0u) | (tok + 1 < lim ? 0xFFFF0000u : 0u);
      }
#pragma unroll
      for (int k = 0; k < D / 64; k++) {
        uint32_t w[4][4];
        v_operands<D, F>(x, vs, k, w);
#pragma unroll
        for (int d = 0; d < 4; d++) {
          const bf16x8 v = operand(w[d][0] & keep[0], w[d][1] & keep[1], w[d][2] & keep[2], w[d][3] & keep[3]);
#pragma unroll
          for (int n = 0; n < NR; n++) {
            const f32x4 o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, pr[n], sum.o[n][4 * k + d], 0, 0, 0);
            const bool mine = lim == (limit[n] < STEP ? limit[n] : STEP);
#pragma unroll
            for (int e = 0; e < 4; e++) sum.o[n][4 * k + d][e] = mine ? o[e] : sum.o[n][4 * k + d][e];
          }
        }
      }
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < D / 64; k++) {
    uint32_t w[4][4];
    v_operands<D, F>(x, vs, k, w);
#pragma unroll
    for (int d = 0; d < 4; d++) {
      const bf16x8 v = operand(w[d][0], w[d][1], w[d][2], w[d][3]);
#pragma unroll
      for (int n = 0; n < NR; n++)
        sum.o[n][4 * k + d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, pr[n], sum.o[n][4 * k + d], 0, 0, 0);
    }
  }
}

template <int D, int F, int NR>
__global__ __launch_bounds__(64 * WAVES, D < 256 && NR == 1 ? 2 : 1) void k_attention(AttnArgs p) {
  __shared__ float ml[WAVES][NR][16][2];
  __shared__ float os[WAVES][16][D + 4];
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x, head = blockIdx.z % p.a.c.heads, b = blockIdx.z / p.a.c.heads;
  const int row0 = blockIdx.y * (16 * NR);
  const int32_t* table = p.a.table + (int64_t)b * p.a.ld_table;
  int len = p.a.lens[b];
  len = len < 0 ? 0 : (int64_t)len > p.a.max_len ? (int)p.a.max_len : len;
  // tokens that a row sees: rows past the last take the last one's
  auto limit_of = [&](int row) {
    row = row < p.rows ? row : p.rows - 1;
    return len - p.a.Lq + 1 + row / p.a.group;
  };
  int lim[NR], end = limit_of(row0 + 16 * NR - 1);
  const int low = limit_of(row0);
#pragma unroll
  for (int n = 0; n < NR; n++) lim[n] = limit_of(row0 + 16 * n + i);
  int t0 = split * p.chunk, t1 = t0 + p.chunk;
  if (t1 > end) t1 = end;
  if (split > 0 && t0 >= t1) return;  // the whole workgroup: no such piece of this request

  const int heads_q = p.a.c.heads * p.a.group;
  bf16x8 q[NR][D / 32];
  Sums<D, NR> sum;
#pragma unroll
  for (int n = 0; n < NR; n++) {
    int row = row0 + 16 * n + i;
    row = row < p.rows ? row : p.rows - 1;
    const int qt = row / p.a.group, hq = head * p.a.group + row - qt * p.a.group;
    const uint16_t* src = p.a.q + ((int64_t)b * p.a.Lq + qt) * p.a.ld_q + (int64_t)hq * D + g * (D / 4);
#pragma unroll
    for (int j = 0; j < D / 32; j++) q[n][j] = *(const bf16x8*)(src + 8 * j);
    sum.m[n] = -__builtin_inff();
    sum.l[n] = 0.0f;
#pragma unroll
    for (int d = 0; d < D / 16; d++) sum.o[n][d] = f32x4{0, 0, 0, 0};
  }
  const float scale2 = p.a.scale * 1.44269504088896340736f;  // scores in units of log 2

  int t = t0 + wave * STEP;
  if (t < t1) {
    Raw<D> x;
    uint32_t there = load_step<D>(p, table, head, t, t1, x);
    while (true) {
      const int next = t + WAVES * STEP;
      Raw<D> ahead;
      uint32_t there_next = 0;
      if (next < t1) there_next = load_step<D>(p, table, head, next, t1, ahead);
      int limit[NR];
#pragma unroll
      for (int n = 0; n < NR; n++) limit[n] = lim[n] - t;
      take_step<D, F, NR>(p, x, q, scale2, there != 3u || t + STEP > low, there, t1 - t, limit, sum);
      t = next;
      if (t >= t1) break;
      x = ahead;
      there = there_next;
    }
  }

  // join the waves
#pragma unroll
  for (int n = 0; n < NR; n++) {
    sum.l[n] = rows_sum(sum.l[n]);
    if (g == 0) {
      ml[wave][n][i][0] = sum.m[n];
      ml[wave][n][i][1] = sum.l[n];
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NR; n++) {
    float m = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < WAVES; w++) m = __builtin_fmaxf(m, ml[w][n][i][0]);
    const float base = m == -__builtin_inff() ? 0.0f : m;
    const float a = __builtin_amdgcn_exp2f(sum.m[n] - base);
#pragma unroll
    for (int d = 0; d < D / 16; d++)
#pragma unroll
      for (int e = 0; e < 4; e++) os[wave][i][(4 * g + e) * (D / 16) + d] = sum.o[n][d][e] * a;
    __syncthreads();
    for (int at = threadIdx.x; at < 16 * D; at += 64 * WAVES) {
      const int r = at / D, d = at % D, row = row0 + 16 * n + r;
      if (row >= p.rows) break;  // later ones are past the last row too
      float mm = -__builtin_inff(), l = 0.0f, o = 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; w++) mm = __builtin_fmaxf(mm, ml[w][n][r][0]);
      const float bb = mm == -__builtin_inff() ? 0.0f : mm;
#pragma unroll
      for (int w = 0; w < WAVES; w++) {
        l += ml[w][n][r][1] * __builtin_amdgcn_exp2f(ml[w][n][r][0] - bb);
        o += os[w][r][d];
      }
      const int qt = row / p.a.group, hq = head * p.a.group + row - qt * p.a.group;
      if (p.splits == 1) {
        const int64_t tok = (int64_t)b * p.a.Lq + qt;
        const bool none = l == 0.0f;  // the row sees no token (the largest score's own p is 1)
        const float v = none ? 0.0f : o / l;
        p.a.o[tok * p.a.ld_o + (int64_t)hq * D + d] = __builtin_bit_cast(uint16_t, (__bf16)v);
        if (d == 0 && p.a.lse)
          p.a.lse[tok * heads_q + hq] = none ? -__builtin_inff() : mm * 0.69314718055994530942f + logf(l);
      } else {
        const int64_t part = (((int64_t)b * p.a.c.heads + head) * p.rows + row) * p.splits + split;
        p.part_o[part * D + d] = o;
        if (d == 0) {
          p.part_ml[2 * part] = mm;
          p.part_ml[2 * part + 1] = l;
        }
      }
    }
    __syncthreads();
  }
}

// Joins the pieces of a row; one wave a row.
template <int D>
__global__ __launch_bounds__(256) void k_attention_join(AttnArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t at = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t total = (int64_t)p.a.B * p.a.c.heads * p.rows;
  if (at >= total) return;
  const int row = (int)(at % p.rows);
  const int64_t bh = at / p.rows;
  const int head = (int)(bh % p.a.c.heads), b = (int)(bh / p.a.c.heads);
  int len = p.a.lens[b];
  len = len < 0 ? 0 : (int64_t)len > p.a.max_len ? (int)p.a.max_len : len;
  const int qt = row / p.a.group, hq = head * p.a.group + row - qt * p.a.group;
  const int limit = len - p.a.Lq + 1 + qt;
  // the pieces that were computed for this row's tile reach past it or end with it
  int n = limit <= 0 ? 0 : (limit + p.chunk - 1) / p.chunk;
  const float* mls = p.part_ml + 2 * at * p.splits;
  float m = -__builtin_inff();
  for (int s = 0; s < n; s++) m = __builtin_fmaxf(m, mls[2 * s]);
  const float base = m == -__builtin_inff() ? 0.0f : m;
  float l = 0.0f, o[D / 64] = {};
  for (int s = 0; s < n; s++) {
    const float a = __builtin_amdgcn_exp2f(mls[2 * s] - base);
    l += mls[2 * s + 1] * a;
#pragma unroll
    for (int k = 0; k < D / 64; k++) o[k] += p.part_o[(at * p.splits + s) * D + 64 * k + lane] * a;
  }
  const int64_t tok = (int64_t)b * p.a.Lq + qt;
#pragma unroll
  for (int k = 0; k < D / 64; k++)
    p.a.o[tok * p.a.ld_o + (int64_t)hq * D + 64 * k + lane] =
        __builtin_bit_cast(uint16_t, (__bf16)(l == 0.0f ? 0.0f : o[k] / l));
  if (lane == 0 && p.a.lse)
    p.a.lse[tok * (p.a.c.heads * p.a.group) + hq] =
        l == 0.0f ? -__builtin_inff() : m * 0.69314718055994530942f + logf(l);
}

// Row tiles of a workgroup, and how the tokens are split: by sizes that the
// host knows, so a result does not depend on timing.
struct Plan {
  int nr, tiles, splits, chunk;
};
Plan plan_of(int64_t B, int64_t Lq, int heads, int group, int dim, int64_t max_len) {
  Plan r;
  const int64_t rows = Lq * group;
  r.nr = rows <= 16 || dim == 256 ? 1 : rows <= 32 || dim == 128 ? 2 : 4;
  r.tiles = (int)((rows + 16 * r.nr - 1) / (16 * r.nr));
  const int64_t unit = STEP * WAVES, base = B * heads * r.tiles;
  const int64_t units = (max_len + unit - 1) / unit;
  int64_t want = (1024 + base - 1) / base;  // four workgroups for each CU
  if (want > (units + 1) / 2) want = (units + 1) / 2;  // at least two steps a wave
  if (want < 1) want = 1;
  int64_t per = (units + want - 1) / want;
  if (per < 1) per = 1;
  r.chunk = (int)(per * unit);
  r.splits = (int)((units + per - 1) / per);
  if (r.splits < 1) r.splits = 1;
  return r;
}

template <int D, int F>
hipError_t attention_by_rows(const AttnArgs& p, const Plan& r, hipStream_t st) {
  const dim3 g((unsigned)r.splits, (unsigned)r.tiles, (unsigned)(p.a.B * p.a.c.heads)), b(64 * WAVES);
  if (r.nr == 1) hipLaunchKernelGGL((k_attention<D, F, 1>), g, b, 0, st, p);
  if constexpr (D <= 128)
    if (r.nr == 2) hipLaunchKernelGGL((k_attention<D, F, 2>), g, b, 0, st, p);
  if constexpr (D == 64)
    if (r.nr == 4) hipLaunchKernelGGL((k_attention<D, F, 4>), g, b, 0, st, p);
  if (r.splits > 1) {
    const int64_t n = (int64_t)p.a.B * p.a.c.heads * p.rows;
    hipLaunchKernelGGL(k_attention_join<D>, dim3((unsigned)((n + 3) / 4)), dim3(256), 0, st, p);
  }
  return hipGetLastError();
}

template <int D>
hipError_t attention_by_fmt(const AttnArgs& p, const Plan& r, hipStream_t st) {
  return p.a.c.fmt == E4M3 ? attention_by_rows<D, E4M3>(p, r, st) : attention_by_rows<D, E5M2>(p, r, st);
}

}  // namespace

hipError_t launch_cache_write(const CacheWriteArgs& a, hipStream_t st) {
  const int64_t n = a.tokens * (2 * a.c.heads * (a.c.dim / 8));
  int64_t blocks = (n + 255) / 256;
  if (blocks > 65536) blocks = 65536;
  const dim3 g((unsigned)blocks), b(256);
  if (a.src == SRC_BF16) {
    if (a.c.fmt == E4M3) hipLaunchKernelGGL((k_cache_write<SRC_BF16, E4M3>), g, b, 0, st, a);
    else hipLaunchKernelGGL((k_cache_write<SRC_BF16, E5M2>), g, b, 0, st, a);
  } else {
    if (a.c.fmt == E4M3) hipLaunchKernelGGL((k_cache_write<SRC_F32, E4M3>), g, b, 0, st, a);
    else hipLaunchKernelGGL((k_cache_write<SRC_F32, E5M2>), g, b, 0, st, a);
  }
  return hipGetLastError();
}

int64_t attention_workspace(int64_t B, int64_t Lq, int heads, int group, int dim, int64_t max_len) {
  const Plan r = plan_of(B, Lq, heads, group, dim, max_len);
  return r.splits == 1 ? 0 : B * heads * Lq * group * r.splits * (dim + 2) * 4;
}

hipError_t launch_attention(const AttentionArgs& a, hipStream_t st) {
  const Plan r = plan_of(a.B, a.Lq, a.c.heads, a.group, a.c.dim, a.max_len);
  AttnArgs p;
  p.a = a;
  p.rows = a.Lq * a.group;
  p.splits = r.splits;
  p.chunk = r.chunk;
  p.page16 = (uint32_t)a.c.page / 16;
  p.magic = p.page16 > 1 ? (uint32_t)(((1ull << 32) + p.page16 - 1) / p.page16) : 0;
  p.part_o = a.work;
  p.part_ml = a.work + (int64_t)a.B * a.c.heads * p.rows * r.splits * a.c.dim;
  switch (a.c.dim) {
    case 64: return attention_by_fmt<64>(p, r, st);
    case 128: return attention_by_fmt<128>(p, r, st);
    default: return attention_by_fmt<256>(p, r, st);
  }
}

}  // namespace mx
