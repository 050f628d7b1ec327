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
// A lane takes 8 elements of a token's head, keys and values (two loads in flight), a
// quad one block.  Bound: HBM; at few tokens the launch.  Tokens of few elements
// share a workgroup.  Measured, 8 heads of dim 128: 8192 tokens, 51 MB, 11.6 us
// (4.4 TB/s; 15.5 with keys and values by different lanes and 64-bit indexes), 32
// tokens 3.0.
template <int SRC, int F>
__device__ __forceinline__ void write_chunk(const uint32_t* raw, uint8_t* q, uint8_t* s, int c) {
  uint32_t v[8], am = 0, rnd[8];
  widen8<SRC>(raw, v);
#pragma unroll
  for (int k = 0; k < 8; k++) am = umax(am, v[k] & 0x7FFFFFFFu);
  am = umax(am, quad_xor1(am));
  am = umax(am, quad_xor2(am));
  const uint32_t code = scale_code<F>(am);
  if ((c & 3) == 0) s[c >> 2] = (uint8_t)code;
  store8<F, false>(q, c, convert8<F, false>(v, code, rnd));
}

template <int SRC, int F>
__global__ __launch_bounds__(256) void k_cache_write(CacheWriteArgs p, int shift, int tokens_per_wg) {
  constexpr int ESZ = SRC == SRC_BF16 ? 2 : 4;
  const int per = p.c.heads << shift;  // chunks of a token's keys; 1 << shift of a head's
  const int sub = tokens_per_wg > 1 ? (int)threadIdx.x / per : 0;
  const int64_t tok = workgroup() * tokens_per_wg + sub;
  if (sub >= tokens_per_wg || tok >= p.tokens) return;
  const int64_t slot = p.slots[tok];  // the same for the lanes of a quad
  if (slot < 0 || slot >= p.c.pages * p.c.page) return;
  const int64_t pg = slot / p.c.page;
  const int at = (int)(slot - pg * p.c.page);
  for (int i = (int)threadIdx.x - sub * per; i < per; i += 256) {
    const int head = i >> shift, c = i & ((1 << shift) - 1);
    uint32_t k[2 * ESZ], v[2 * ESZ];
    load_elems<ESZ, 8, false>((const uint8_t*)p.k + tok * p.ld_k + head * p.hs_k + c * 8 * ESZ, 8, k);
    load_elems<ESZ, 8, false>((const uint8_t*)p.v + tok * p.ld_v + head * p.hs_v + c * 8 * ESZ, 8, v);
    const int64_t row = (pg * p.c.heads + head) * p.c.page + at;
    write_chunk<SRC, F>(k, p.c.k_q + row * p.c.dim, p.c.k_s + row * (p.c.dim / 32), c);
    write_chunk<SRC, F>(v, p.c.v_q + row * p.c.dim, p.c.v_s + row * (p.c.dim / 32), c);
  }
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
// Rows of a key/value head are its (query token, query head) pairs.  Up to 16 of them:
// a workgroup takes them all and one piece of the request's tokens, each wave 32
// tokens at a time.  Both products run on 16x16x32 bf16 matrix instructions, to which
// an element times its scale is exact from bf16's smallest normal value, 2^-126, on:
//   S^T = K Q^T   lane (l % 16, g = l / 16) takes dims g D/4 .. of token l % 16 and
//                 feeds dims 8 j .. of them to instruction j, as the lane of Q does;
//                 it gets its row's scores of tokens 4 g .. 4 g + 3
//   O^T = V^T P^T those 8 scores (two groups of 16 tokens) are the lane's 8 of the
//                 32 of a sum over tokens as they are; the lane takes dims
//                 (l % 16) D/16 .. of the same 8 tokens and transposes 2 x 2
// so P stays in registers, as two bf16 terms (see `weights`); scores, maxima, sums and
// O stay in fp32.
//
// Bound for a few rows: HBM, 2 (D + D / 32) bytes a token and head.  Each wave loads
// its 32 tokens in whole 1 KB runs and reads them again from its own piece of LDS:
// with loads in the operands' order (16 bytes of a token 32 bytes apart, scales byte
// by byte) 32 requests to 16384 took 165 us, 136 us this way, and 140 us with weights of
// two terms (661 MB: 4.7 TB/s).  The next 32 tokens are in flight meanwhile.  What is
// lost there: a CU holds a wave in 62 % of the time only (the large norm: 90 %).
// Workgroups go to the eight XCDs by turns, so with 4 pieces piece p is always on XCDs
// p and p + 4, and while every request has a first piece, few have a last one.
constexpr int STEP = 32;  // tokens a wave takes at a time

struct AttnArgs {
  AttentionArgs a;
  int rows;              // Lq * group
  int splits;
  int chunk;             // tokens of a piece, a multiple of what its waves take at a time
  uint32_t page16, magic, shift;  // page / 16 and the constants that divide by it
  // sums and (base, l) of the pieces: by rows [B][heads][rows][splits][dim] and [2], or
  // by tiles of 16 rows [B][heads][tiles][splits][dim / 16][64 lanes][4] and [16][2]
  float *part_o, *part_ml;
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

// The bytes of 32 tokens in a lane: in 16-byte pieces of each group of 16 tokens in
// the order of the cache, and the scales of token l % 16, keys of the first and of
// the second group, then values.
template <int D>
struct Raw {
  u32x4 k[2][D / 64], v[2][D / 64];
  uint32_t s[D == 256 ? 2 : 1];
};
// A wave's piece of LDS: rows of keys, of values and of scales, with pitches that
// spread the lanes' reads over the banks.
template <int D>
struct Stage {
  static constexpr int KP = D + 16, VP = D == 128 ? 160 : D + 16, SP = D / 32;
  static constexpr int K_AT = 0, V_AT = K_AT + 32 * KP, KS_AT = V_AT + 32 * VP, VS_AT = KS_AT + 32 * SP;
  static constexpr int BYTES = VS_AT + 32 * SP;
};

// i / page16 for i < 2^27: with 2^(L - 1) < page16 <= 2^L, the constant c =
// ceil(2^(27 + L) / page16) is too large by less than 1, so i c / 2^(27 + L) by less
// than 1 / 2^L <= 1 / page16.  magic is 16 c, which has 32 bits, and shift L - 1.
__device__ __forceinline__ uint32_t page_index(const AttnArgs& p, uint32_t i) {
  return p.page16 == 1 ? i : __umulhi(i, p.magic) >> p.shift;
}

// The page of tokens t0 + 16 (l & 1) .. of a request in lane l, -1 where there are
// none.  By a vector load and a step ahead of its use: a wave that waits for a page
// number before it can load tokens does nothing else meanwhile.
__device__ __forceinline__ int page_of(const AttnArgs& p, const int32_t* table, int t0, int end) {
  const int tok = t0 + 16 * (int)(threadIdx.x & 1);
  if (tok >= end) return -1;
  const uint32_t i16 = (uint32_t)tok >> 4;
  return table[page_index(p, i16)];
}
// Row (page, head, place) of the cache at which tokens t0 + 16 u .. begin.  A page
// that is not one of the cache's holds no tokens; any row stands in for it, and what
// it holds is masked.
__device__ __forceinline__ bool locate(const AttnArgs& p, int pages, int head, int t0, int u, int64_t& row) {
  const int pg = __builtin_amdgcn_readlane(pages, u);
  const uint32_t i16 = (uint32_t)(t0 + 16 * u) >> 4;
  const uint32_t idx = page_index(p, i16);
  const bool ok = (uint32_t)pg < (uint32_t)p.a.c.pages;
  row = ok ? ((int64_t)pg * p.a.c.heads + head) * p.a.c.page + (int)(i16 - idx * p.page16) * 16 : 0;
  return ok;
}

template <int D>
__device__ __forceinline__ uint32_t load_step(const AttnArgs& p, int pages, int head, int t0,
                                              Raw<D>& x) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t there = 0;
  int64_t row[2];
#pragma unroll
  for (int u = 0; u < 2; u++) {
    const bool ok = locate(p, pages, head, t0, u, row[u]);
    there |= (uint32_t)ok << u;
  }
#pragma unroll
  for (int u = 0; u < 2; u++)
#pragma unroll
    for (int c = 0; c < D / 64; c++) {
      x.k[u][c] = *(const u32x4*)(p.a.c.k_q + row[u] * D + (1024 * c + 16 * lane));
      x.v[u][c] = *(const u32x4*)(p.a.c.v_q + row[u] * D + (1024 * c + 16 * lane));
    }
  const uint8_t* s = (lane & 32 ? p.a.c.v_s : p.a.c.k_s) + ((lane & 16 ? row[1] : row[0]) + (lane & 15)) * (D / 32);
  if constexpr (D == 64) x.s[0] = *(const uint16_t*)s;
  else load_words<D / 128>(s, x.s);
  return there;
}

// Into the wave's piece of LDS.  `cut`: tokens at or past `end` or not there may be
// among them; they count as zeros whatever the cache holds there, for 0 * NaN is
// not 0.  True where a value of the others may not be finite (asked only then).
template <int D, int F>
__device__ __forceinline__ bool stage_step(Raw<D>& x, uint8_t* lds, bool cut, uint32_t there, int end) {
  using St = Stage<D>;
  const int lane = threadIdx.x & 63;
  bool odd = false;
  if (cut) {
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
      for (int c = 0; c < D / 64; c++) {
        const int tok = 16 * u + (64 * c + lane) / (D / 16);
        const bool gone = !(there >> u & 1) || tok >= end;
        const u32x4 v = gone ? u32x4{0, 0, 0, 0} : x.v[u][c];
        x.v[u][c] = v;
        constexpr uint32_t add = F == E4M3 ? 0x01010101u : 0x04040404u;  // to the sign bit: NaN, or Inf and NaN
        odd |= ((((v.x & 0x7F7F7F7Fu) + add) | ((v.y & 0x7F7F7F7Fu) + add) | ((v.z & 0x7F7F7F7Fu) + add) |
                 ((v.w & 0x7F7F7F7Fu) + add)) & 0x80808080u) != 0;
      }
    if (lane & 32) {
      const int u = (lane >> 4) & 1;
      const bool gone = !(there >> u & 1) || 16 * u + (lane & 15) >= end;
#pragma unroll
      for (int c = 0; c < (D == 256 ? 2 : 1); c++) {
        if (gone) x.s[c] = 0x7F7F7F7Fu;
#pragma unroll
        for (int k = 0; k < (D == 64 ? 2 : 4); k++) odd |= ((x.s[c] >> (8 * k)) & 0xFFu) > (uint32_t)(254 - Fmt<F>::emax);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < 2; u++)
#pragma unroll
    for (int c = 0; c < D / 64; c++) {
      const int f = 64 * c + lane, tok = 16 * u + f / (D / 16), at = f % (D / 16) * 16;
      *(u32x4*)(lds + St::K_AT + tok * St::KP + at) = x.k[u][c];
      *(u32x4*)(lds + St::V_AT + tok * St::VP + at) = x.v[u][c];
    }
  uint8_t* s = lds + St::KS_AT + lane * St::SP;  // keys 0 .. 31, values 0 .. 31
  if constexpr (D == 64) *(uint16_t*)s = (uint16_t)x.s[0];
  else if constexpr (D == 128) *(uint32_t*)s = x.s[0];
  else *(uint2*)s = make_uint2(x.s[0], x.s[1]);
  return odd;
}
// lanes of one wave: what one wrote to LDS, the others read
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ bf16x8 operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8, make_uint4(a, b, c, d));
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// V as operands of the second product: dims (l % 16) D/16 + 4 k .. + 3 of the
// lane's 8 tokens, 16 u + 4 g + r (dword c of an operand: tokens 2 c and 2 c + 1).
template <int D, int F>
__device__ __forceinline__ void v_operands(const uint8_t* lds, int k, uint32_t (&w)[4][4]) {
  using St = Stage<D>;
  const int i = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int u = 0; u < 2; u++)
#pragma unroll
    for (int h = 0; h < 2; h++) {
      uint32_t raw[2];
      float s[2];
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const int tok = 16 * u + 4 * g + 2 * h + e;
        raw[e] = *(const uint32_t*)(lds + St::V_AT + tok * St::VP + i * (D / 16) + 4 * k);
        s[e] = e8m0(lds[St::VS_AT + tok * St::SP + i * (D / 16) / 32]);
      }
      const uint32_t a0 = cvt_lo<F>(raw[0], s[0]), a1 = cvt_hi<F>(raw[0], s[0]);
      const uint32_t b0 = cvt_lo<F>(raw[1], s[1]), b1 = cvt_hi<F>(raw[1], s[1]);
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

// Weights of a step as operands of the second product: p is the sum of two bf16 terms.
// hi is p cut to 8 bits; lo is what is left of it, and 2^-20 p, rounded: p is kept to
// 2^-15 (one rounded term would leave 2^-8 of each weight, as much as the output's own
// rounding).  lo is above zero where p is, so an infinite value stays one.  Measured (us,
// one rounded term / these two): 32 requests to 16384 136 / 140, 1 of 1000 10.9 / 11.3;
// where rows share tokens, 4 requests of 64 query tokens to 4096 27.2 / 28.7, two
// prompts of 2048 128 / 147, by the second products and 24 more instructions for 8 weights.
struct Weights {
  bf16x8 hi, lo;
};
__device__ __forceinline__ Weights weights(const f32x4 (&p)[2]) {
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int k = 0; k < 4; k++) {
    const float v0 = p[k >> 1][2 * (k & 1)], v1 = p[k >> 1][2 * (k & 1) + 1];
    const uint32_t u0 = __builtin_bit_cast(uint32_t, v0), u1 = __builtin_bit_cast(uint32_t, v1);
    hi[k] = __builtin_amdgcn_perm(u1, u0, 0x07060302u);
    lo[k] = bf16_pair(__builtin_fmaf(v0, 1.0f + 0x1p-20f, -__builtin_bit_cast(float, u0 & 0xFFFF0000u)),
                      __builtin_fmaf(v1, 1.0f + 0x1p-20f, -__builtin_bit_cast(float, u1 & 0xFFFF0000u)));
  }
  return {operand(hi[0], hi[1], hi[2], hi[3]), operand(lo[0], lo[1], lo[2], lo[3])};
}

// Maxima, weights and sums of a step's scores (in units of log 2, masked); the weights
// p take the scores' place.  The base that scores are taken from is a maximum of
// earlier ones: it moves, and the sums with it, only where a score passes it by more
// than 8, so p stays below 2^8 and O is seldom multiplied.  o / l does not depend on
// the base.
template <int D, int NR>
__device__ __forceinline__ void soften(f32x4 (&s)[NR][2], Sums<D, NR>& sum) {
#pragma unroll
  for (int n = 0; n < NR; n++) {
    float v[8], top = -__builtin_inff();
#pragma unroll
    for (int e = 0; e < 8; e++) {
      v[e] = s[n][e >> 2][e & 3];
      top = __builtin_fmaxf(top, v[e]);
    }
    top = rows_max(top);
    if (__any(top > sum.m[n] + 8.0f)) {
      const float m = __builtin_fmaxf(sum.m[n], top);
      const float a = __builtin_amdgcn_exp2f(sum.m[n] - (m == -__builtin_inff() ? 0.0f : m));
      sum.m[n] = m;
      sum.l[n] *= a;
#pragma unroll
      for (int d = 0; d < D / 16; d++) sum.o[n][d] *= a;
    }
    const float base = sum.m[n] == -__builtin_inff() ? 0.0f : sum.m[n];  // nothing seen yet: every p is 0
#pragma unroll
    for (int e = 0; e < 8; e++) {
      v[e] = __builtin_amdgcn_exp2f(v[e] - base);
      sum.l[n] += v[e];
      s[n][e >> 2][e & 3] = v[e];
    }
  }
}

// One step of 32 staged tokens.  `cut`: some row does not see all of them, or some
// are not there.  `limit` is the number of them that the lane's row sees (less than 1:
// none, 32 or more: all).  `odd`: values may not be finite and rows see different
// tokens.
template <int D, int F>
__device__ __forceinline__ void take_step(uint8_t* lds, const bf16x8 (*q)[64], float scale2, bool cut,
                                          bool odd, uint32_t there, int limit, Sums<D, 1>& sum) {
  using St = Stage<D>;
  const int i = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  f32x4 s[1][2] = {{f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}}};
#pragma unroll
  for (int c = 0; c < D / 64; c++) {  // 16 bytes: dims g D/4 + 16 c .. of token 16 u + i
    uint4 kw[2];
    float ks[2];
#pragma unroll
    for (int u = 0; u < 2; u++) {
      kw[u] = *(const uint4*)(lds + St::K_AT + (16 * u + i) * St::KP + g * (D / 4) + 16 * c);
      ks[u] = e8m0(lds[St::KS_AT + (16 * u + i) * St::SP + (g * (D / 4) + 16 * c) / 32]);
    }
#pragma unroll
    for (int h = 0; h < 2; h++) {
      bf16x8 k[2];
#pragma unroll
      for (int u = 0; u < 2; u++) {
        const uint32_t w0 = h ? kw[u].z : kw[u].x, w1 = h ? kw[u].w : kw[u].y;
        k[u] = operand(cvt_lo<F>(w0, ks[u]), cvt_hi<F>(w0, ks[u]), cvt_lo<F>(w1, ks[u]), cvt_hi<F>(w1, ks[u]));
      }
      const bf16x8 qj = q[2 * c + h][threadIdx.x & 63];
#pragma unroll
      for (int u = 0; u < 2; u++) s[0][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[u], qj, s[0][u], 0, 0, 0);
    }
  }
#pragma unroll
  for (int u = 0; u < 2; u++) s[0][u] *= scale2;
  if (cut) {  // after the scaling, whose sign is the caller's
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const int tok = 16 * (e >> 2) + 4 * g + (e & 3);
      const bool seen = tok < limit && (there >> (e >> 2) & 1);
      s[0][e >> 2][e & 3] = seen ? s[0][e >> 2][e & 3] : -__builtin_inff();
    }
  }
  soften<D, 1>(s, sum);
  if (odd) {
    // 0 * NaN is not 0: token by token, for the rows that see it.  p takes the
    // place of the keys.
    wave_fence();
    float* ps = (float*)(lds + St::K_AT);  // [row][token]
    static_assert(32 * St::KP >= 16 * STEP * 4, "weights fit into the keys' place");
    *(f32x4*)(ps + STEP * i + 4 * g) = s[0][0];
    *(f32x4*)(ps + STEP * i + 16 + 4 * g) = s[0][1];
    wave_fence();
    for (int tok = 0; tok < STEP; tok++) {
      if (tok >= limit) continue;
      const float pt = ps[STEP * i + tok];
#pragma unroll
      for (int e = 0; e < 4; e++)
#pragma unroll
        for (int k = 0; k < D / 64; k++) {
          const int at = (4 * g + e) * (D / 16) + 4 * k;  // dims at .. at + 3
          const uint32_t raw = *(const uint32_t*)(lds + St::V_AT + tok * St::VP + at);
          const float sc = e8m0(lds[St::VS_AT + tok * St::SP + at / 32]);
          const uint32_t a = cvt_lo<F>(raw, sc), b = cvt_hi<F>(raw, sc);
#pragma unroll
          for (int d = 0; d < 4; d++) {
            const uint32_t h = d < 2 ? a : b;
            const float v = __builtin_bit_cast(float, d & 1 ? h & 0xFFFF0000u : h << 16);
            sum.o[0][4 * k + d][e] = __builtin_fmaf(pt, v, sum.o[0][4 * k + d][e]);
          }
        }
    }
    return;
  }
  const Weights pr = weights(s[0]);
#pragma unroll
  for (int k = 0; k < D / 64; k++) {
    uint32_t w[4][4];
    v_operands<D, F>(lds, k, w);
#pragma unroll
    for (int e = 0; e < 2; e++)
#pragma unroll
      for (int d = 0; d < 4; d++) {
        const bf16x8 v = operand(w[d][0], w[d][1], w[d][2], w[d][3]);
        sum.o[0][4 * k + d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, e ? pr.lo : pr.hi, sum.o[0][4 * k + d], 0, 0, 0);
      }
  }
}

template <int D, int F, int WAVES, int OCC>
__global__ __launch_bounds__(64 * WAVES, OCC) void k_attention(AttnArgs p) {
  __shared__ float ml[WAVES][16][2];
  // the waves' staged tokens, then their outputs
  constexpr int OS = 4 * 16 * (D + 4), PIECE = Stage<D>::BYTES > OS ? Stage<D>::BYTES : OS;
  __shared__ __align__(16) uint8_t lds[WAVES * PIECE];
  float(*os)[16][D + 4] = (float(*)[16][D + 4])lds;
  __shared__ bf16x8 q[D / 32][64];  // by lane, the same for every wave
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x, head = blockIdx.y % p.a.c.heads, b = blockIdx.y / p.a.c.heads;
  const int32_t* table = p.a.table + (int64_t)b * p.a.ld_table;
  int len = p.a.lens[b];
  len = len < 0 ? 0 : (int64_t)len > p.a.max_len ? (int)p.a.max_len : len;
  const int row = i < p.rows ? i : p.rows - 1;  // lanes past the last row repeat it
  const int qt = row / p.a.group, hq = head * p.a.group + row - qt * p.a.group;
  const int low = len - p.a.Lq + 1, lim = low + qt, end = low + (p.rows - 1) / p.a.group;  // tokens that rows see
  int t0 = split * p.chunk, t1 = t0 + p.chunk;
  if (t1 > end) t1 = end;
  if (split > 0 && t0 >= t1) return;  // the whole workgroup: no such piece of this request

  Sums<D, 1> sum;
  const uint16_t* src = p.a.q + ((int64_t)b * p.a.Lq + qt) * p.a.ld_q + (int64_t)hq * D + g * (D / 4);
  for (int j = wave; j < D / 32; j += WAVES) q[j][lane] = *(const bf16x8*)(src + 8 * j);
  sum.m[0] = -__builtin_inff();
  sum.l[0] = 0.0f;
#pragma unroll
  for (int d = 0; d < D / 16; d++) sum.o[0][d] = f32x4{0, 0, 0, 0};
  __syncthreads();
  const float scale2 = p.a.scale * 1.44269504088896340736f;  // scores in units of log 2

  int t = t0 + wave * STEP;
  if (t < t1) {
    uint8_t* mine = lds + wave * Stage<D>::BYTES;
    Raw<D> x;
    constexpr int STRIDE = WAVES * STEP;
    uint32_t there = load_step<D>(p, page_of(p, table, t, t1), head, t, x);
    int pages = page_of(p, table, t + STRIDE, t1);
    while (true) {
      const bool cut = there != 3u || t + STEP > low;
      const uint32_t here = there;
      const bool odd = __any(stage_step<D, F>(x, mine, cut, here, t1 - t)) && p.a.Lq > 1;
      wave_fence();
      const int next = t + STRIDE;
      if (next < t1) {
        there = load_step<D>(p, pages, head, next, x);
        pages = page_of(p, table, next + STRIDE, t1);
      }
      take_step<D, F>(mine, q, scale2, cut, odd, here, lim - t, sum);
      wave_fence();
      t = next;
      if (t >= t1) break;
    }
  }

  // join the waves
  sum.l[0] = rows_sum(sum.l[0]);
  if (g == 0) {
    ml[wave][i][0] = sum.m[0];
    ml[wave][i][1] = sum.l[0];
  }
  __syncthreads();  // the staged tokens' place holds outputs now
  float m = -__builtin_inff();
#pragma unroll
  for (int w = 0; w < WAVES; w++) m = __builtin_fmaxf(m, ml[w][i][0]);
  const float a = __builtin_amdgcn_exp2f(sum.m[0] - (m == -__builtin_inff() ? 0.0f : m));
#pragma unroll
  for (int d = 0; d < D / 16; d++)
#pragma unroll
    for (int e = 0; e < 4; e++) os[wave][i][(4 * g + e) * (D / 16) + d] = sum.o[0][d][e] * a;
  __syncthreads();
  for (int at = threadIdx.x; at < p.rows * D; at += 64 * WAVES) {
    const int r = at / D, d = at % D;
    float mm = -__builtin_inff(), l = 0.0f, o = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; w++) mm = __builtin_fmaxf(mm, ml[w][r][0]);
    const float base = mm == -__builtin_inff() ? 0.0f : mm;
#pragma unroll
    for (int w = 0; w < WAVES; w++) {
      l += ml[w][r][1] * __builtin_amdgcn_exp2f(ml[w][r][0] - base);
      o += os[w][r][d];
    }
    if (p.splits == 1) {
      const int rt = r / p.a.group;
      const int64_t tok = (int64_t)b * p.a.Lq + rt, hr = head * p.a.group + r - rt * p.a.group;
      const bool none = l == 0.0f;  // the row sees no token (the largest score's own p is not 0)
      p.a.o[tok * p.a.ld_o + hr * D + d] = __builtin_bit_cast(uint16_t, (__bf16)(none ? 0.0f : o / l));
      if (d == 0 && p.a.lse)
        p.a.lse[tok * (p.a.c.heads * p.a.group) + hr] =
            none ? -__builtin_inff() : mm * 0.69314718055994530942f + logf(l);
    } else {
      const int64_t part = (((int64_t)b * p.a.c.heads + head) * p.rows + r) * p.splits + split;
      p.part_o[part * D + d] = o;
      if (d == 0) {
        p.part_ml[2 * part] = mm;
        p.part_ml[2 * part + 1] = l;
      }
    }
  }
}

// Many rows: the waves of a workgroup take 16 NR rows each and share the tokens, 32
// at a time, so a token is converted once for 64 NR rows.  The workgroup converts
// its tokens to bf16 into LDS, in two buffers by turns (one barrier a step), while
// the next ones are on their way:
//   K  [token][dims], 16 more bytes a row
//   V  [dim][token] with the dims that a lane holds (4 c .. 4 c + 3) D/4 rows apart
//      (row_of), tokens in the order of the second product's lanes (8 g + 4 u + r for
//      token 16 u + 4 g + r), and the four 16-byte pieces of a row exchanged by row, so
//      that both the writes and the reads spread over the banks
// Bound: by no unit, but by waves that wait and by CUs that stand empty.  4 requests of 64
// query tokens to 4096, 8 heads and 32 query heads, D = 128, take 29 us and 7.4 us for
// the join.  Of the 29 us the matrix units are busy for 13 %, vector instructions issue
// for 22 %, and a CU holds a wave for 58 %: the pieces are cut by max_len, so shorter
// requests have fewer, and a workgroup has 8 steps at most beside a beginning (length,
// page, tokens: 6000 cycles) and an end (2500); the join reads 29 MB of partial sums
// again.  Two prompts of up to 2048, 147 us: 16 %, 25 % and 55 %.
// Tried without gain: all reads of a step ahead of their use, scores scaled in the
// exponent's subtraction, the first tokens loaded before the request's length is known.
template <int D>
struct Shared {
  static constexpr int KP = 2 * D + 16, K_BYTES = 32 * KP, BYTES = K_BYTES + D * 64;
  static constexpr int KL = D <= 128 ? 1 : D / 128;           // 16-byte pieces of K in a lane
  static constexpr int VL = KL;                               // 4 x 4 pieces of V in a lane
  static constexpr int USED = D < 128 ? 2 * D : 256;          // lanes that hold pieces
  __device__ static int v_at(int row, int piece) { return K_BYTES + row * 64 + ((piece ^ (row >> 2)) & 3) * 16; }
};
template <int D>
struct Tokens {
  u32x4 k[Shared<D>::KL];
  uint32_t ks[Shared<D>::KL];
  uint32_t v[Shared<D>::VL][4], vs[Shared<D>::VL][D / 32];
};

template <int D>
__device__ __forceinline__ uint32_t load_tokens(const AttnArgs& p, int pages, int head, int t0,
                                                Tokens<D>& x) {
  const int tid = threadIdx.x;
  uint32_t there = 0;
  int64_t row[2];
#pragma unroll
  for (int u = 0; u < 2; u++) {
    const bool ok = locate(p, pages, head, t0, u, row[u]);
    there |= (uint32_t)ok << u;
  }
  if (Shared<D>::USED < 256 && tid >= Shared<D>::USED) return there;
#pragma unroll
  for (int c = 0; c < Shared<D>::KL; c++) {
    const int f = tid + 256 * c, tok = f / (D / 16), at = f % (D / 16);
    const int64_t r = (tok < 16 ? row[0] : row[1]) + (tok & 15);
    x.k[c] = *(const u32x4*)(p.a.c.k_q + r * D + 16 * at);
    x.ks[c] = p.a.c.k_s[r * (D / 32) + at / 2];
    const int quad = f / (D / 4), dc = f % (D / 4);  // tokens 4 quad .., dims 4 dc ..
    const int64_t rv = (quad < 4 ? row[0] : row[1]) + 4 * (quad & 3);
#pragma unroll
    for (int r4 = 0; r4 < 4; r4++) x.v[c][r4] = *(const uint32_t*)(p.a.c.v_q + (rv + r4) * D + 4 * dc);
    load_words<D / 32>(p.a.c.v_s + rv * (D / 32), x.vs[c]);
  }
  return there;
}

// Converted into a buffer; tokens that are cut are zeros (stage_step says why).  True
// where another value may not be finite (asked only with `cut`).
template <int D, int F>
__device__ __forceinline__ bool stage_tokens(const Tokens<D>& x, uint8_t* buf, bool cut, uint32_t there, int end) {
  using Sh = Shared<D>;
  const int tid = threadIdx.x;
  bool odd = false;
  if (Sh::USED < 256 && tid >= Sh::USED) return odd;
#pragma unroll
  for (int c = 0; c < Sh::KL; c++) {
    const int f = tid + 256 * c;
    const float ks = e8m0(x.ks[c]);
    uint8_t* kd = buf + f / (D / 16) * Sh::KP + f % (D / 16) * 32;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const uint32_t w0 = x.k[c][2 * h], w1 = x.k[c][2 * h + 1];
      *(u32x4*)(kd + 16 * h) = u32x4{cvt_lo<F>(w0, ks), cvt_hi<F>(w0, ks), cvt_lo<F>(w1, ks), cvt_hi<F>(w1, ks)};
    }
    const int quad = f / (D / 4), dc = f % (D / 4), blk = dc / 8;
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int r = 0; r < 4; r++) {
      // byte r D/32 + blk of x.vs[c]
      uint32_t code, raw = x.v[c][r];
      if constexpr (D == 64) code = (x.vs[c][r >> 1] >> (16 * (r & 1) + 8 * blk)) & 0xFFu;
      else if constexpr (D == 128) code = (x.vs[c][r] >> (8 * blk)) & 0xFFu;
      else code = ((blk & 4 ? x.vs[c][2 * r + 1] : x.vs[c][2 * r]) >> (8 * (blk & 3))) & 0xFFu;
      if (cut) {
        const bool gone = !(there >> (quad >> 2) & 1) || 4 * quad + r >= end;
        code = gone ? 127u : code;
        raw = gone ? 0u : raw;
        odd |= (((raw & 0x7F7F7F7Fu) + (F == E4M3 ? 0x01010101u : 0x04040404u)) & 0x80808080u) != 0 ||
               code > (uint32_t)(254 - Fmt<F>::emax);
      }
      lo[r] = cvt_lo<F>(raw, e8m0(code));
      hi[r] = cvt_hi<F>(raw, e8m0(code));
    }
    const int piece = quad & 3, half = 8 * (quad >> 2);
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const uint32_t* w = e < 2 ? lo : hi;
      const uint32_t sel = e & 1 ? 0x07060302u : 0x05040100u;
      *(uint2*)(buf + Sh::v_at(e * (D / 4) + dc, piece) + half) =
          make_uint2(__builtin_amdgcn_perm(w[1], w[0], sel), __builtin_amdgcn_perm(w[3], w[2], sel));
    }
  }
  return odd;
}

// Outputs of the 16 rows from row0 on.  ND pieces of the sums as the second product
// leaves them (piece d0 + d of row l % 16), divided by the row's l, go to `os`, 16
// (D + 2) bf16 of LDS; `count` waves then store the rows, this one from `first` on.
template <int D, int ND>
__device__ __forceinline__ void put_rows(const f32x4 (&o)[ND], int d0, float l, uint16_t* os) {
  const int i = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // l = 0: the row sees no token
#pragma unroll
  for (int d = 0; d < ND; d++)
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const int r = 16 * (d0 + d) + 4 * g + e;  // row of V's buffer: dim 4 (r % (D / 4)) + r / (D / 4)
      os[i * (D + 2) + 4 * (r % (D / 4)) + r / (D / 4)] = __builtin_bit_cast(uint16_t, (__bf16)(o[d][e] * inv));
    }
}
template <int D>
__device__ __forceinline__ void store_rows(const AttnArgs& p, int b, int head, int row0, float l, float m,
                                           const uint16_t* os, int first, int count) {
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int row = row0 + i, qt = row / p.a.group, hq = head * p.a.group + row - qt * p.a.group;
  if (first == 0 && g == 0 && row < p.rows && p.a.lse)
    p.a.lse[((int64_t)b * p.a.Lq + qt) * (p.a.c.heads * p.a.group) + hq] =
        l == 0.0f ? -__builtin_inff() : m * 0.69314718055994530942f + logf(l);
#pragma unroll 4
  for (int r = first; r < 16; r += count) {
    if (row0 + r >= p.rows) break;
    const int64_t tok = (int64_t)b * p.a.Lq + __builtin_amdgcn_readlane(qt, r);
    uint16_t* to = p.a.o + tok * p.a.ld_o + (int64_t)__builtin_amdgcn_readlane(hq, r) * D;
#pragma unroll
    for (int k = 0; k < D / 64; k++) to[64 * k + lane] = os[r * (D + 2) + 64 * k + lane];
  }
}

template <int D, int F, int NR>
__global__ __launch_bounds__(256, 2) void k_attention_rows(AttnArgs p) {
  using Sh = Shared<D>;
  constexpr int OS = 16 * (D + 2) * 2;  // bytes of a wave's 16 rows of outputs
  static_assert(2 * Sh::BYTES >= 4 * OS, "outputs fit into the buffers");
  __shared__ __align__(16) uint8_t lds[2 * Sh::BYTES];
  __shared__ __align__(16) float ps[4][16][STEP];
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x, head = blockIdx.y % p.a.c.heads, b = blockIdx.y / p.a.c.heads;
  // the last rows see most tokens: their workgroups begin first
  const int wg0 = (int)(gridDim.z - 1 - blockIdx.z) * (64 * NR), row0 = wg0 + wave * (16 * NR);
  const int32_t* table = p.a.table + (int64_t)b * p.a.ld_table;
  int len = p.a.lens[b];
  len = len < 0 ? 0 : (int64_t)len > p.a.max_len ? (int)p.a.max_len : len;
  auto limit_of = [&](int row) {  // tokens that a row sees: rows past the last take the last one's
    row = row < p.rows ? row : p.rows - 1;
    return len - p.a.Lq + 1 + row / p.a.group;
  };
  int t0 = split * p.chunk, t1 = t0 + p.chunk;
  const int end = limit_of(wg0 + 64 * NR - 1);
  if (t1 > end) t1 = end;
  if (split > 0 && t0 >= t1) return;  // the whole workgroup: no such piece of this request
  const int low = limit_of(wg0), wave_low = limit_of(row0), wave_end = limit_of(row0 + 16 * NR - 1);
  const bool idle = row0 >= p.rows;

  bf16x8 q[NR][D / 32];
  Sums<D, NR> sum;
  int lim[NR];
#pragma unroll
  for (int n = 0; n < NR; n++) {
    int row = row0 + 16 * n + i;
    lim[n] = limit_of(row);
    row = row < p.rows ? row : p.rows - 1;
    const int qt = row / p.a.group, hq = head * p.a.group + row - qt * p.a.group;
    const uint16_t* src = p.a.q + ((int64_t)b * p.a.Lq + qt) * p.a.ld_q + (int64_t)hq * D + 8 * g;
#pragma unroll
    for (int j = 0; j < D / 32; j++) q[n][j] = *(const bf16x8*)(src + 32 * j);
    sum.m[n] = -__builtin_inff();
    sum.l[n] = 0.0f;
#pragma unroll
    for (int d = 0; d < D / 16; d++) sum.o[n][d] = f32x4{0, 0, 0, 0};
  }
  const float scale2 = p.a.scale * 1.44269504088896340736f;  // scores in units of log 2

  Tokens<D> x;
  uint32_t there = 0;
  int pages = -1;
  if (t0 < t1) {
    there = load_tokens<D>(p, page_of(p, table, t0, t1), head, t0, x);
    pages = page_of(p, table, t0 + STEP, t1);
  }
  for (int t = t0, turn = 0; t < t1; t += STEP, turn ^= 1) {
    uint8_t* buf = lds + turn * Sh::BYTES;
    const uint32_t here = there;
    const bool wg_cut = here != 3u || t + STEP > low;
    bool odd = stage_tokens<D, F>(x, buf, wg_cut, here, t1 - t);
    if (wg_cut) odd = __syncthreads_or(odd) != 0;
    else __syncthreads();
    if (t + STEP < t1) {
      there = load_tokens<D>(p, pages, head, t + STEP, x);
      pages = page_of(p, table, t + 2 * STEP, t1);
    }
    if (idle || t >= wave_end) continue;
    f32x4 s[NR][2];
#pragma unroll
    for (int n = 0; n < NR; n++) s[n][0] = s[n][1] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < D / 32; j++)
#pragma unroll
      for (int u = 0; u < 2; u++) {
        const bf16x8 k = *(const bf16x8*)(buf + (16 * u + i) * Sh::KP + 64 * j + 16 * g);
#pragma unroll
        for (int n = 0; n < NR; n++) s[n][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[n][j], s[n][u], 0, 0, 0);
      }
#pragma unroll
    for (int n = 0; n < NR; n++)
#pragma unroll
      for (int u = 0; u < 2; u++) s[n][u] *= scale2;
    if (here != 3u || t + STEP > wave_low) {
#pragma unroll
      for (int n = 0; n < NR; n++)
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const int tok = 16 * (e >> 2) + 4 * g + (e & 3);
          const bool seen = tok < lim[n] - t && (here >> (e >> 2) & 1);
          s[n][e >> 2][e & 3] = seen ? s[n][e >> 2][e & 3] : -__builtin_inff();
        }
    }
    soften<D, NR>(s, sum);
    if (odd && p.a.Lq > 1) {
      // 0 * NaN is not 0: token by token, for the rows that see it
#pragma unroll
      for (int n = 0; n < NR; n++) {
        wave_fence();
        *(f32x4*)&ps[wave][i][4 * g] = s[n][0];
        *(f32x4*)&ps[wave][i][16 + 4 * g] = s[n][1];
        wave_fence();
        for (int tok = 0; tok < STEP; tok++) {
          if (tok >= lim[n] - t) continue;
          const float pt = ps[wave][i][tok];
#pragma unroll
          for (int d = 0; d < D / 16; d++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const uint16_t v = *(const uint16_t*)(buf + Sh::v_at(16 * d + 4 * g + e, (tok & 15) >> 2) +
                                                    8 * (tok >> 4) + 2 * (tok & 3));
              sum.o[n][d][e] = __builtin_fmaf(pt, __builtin_bit_cast(float, (uint32_t)v << 16), sum.o[n][d][e]);
            }
        }
      }
      continue;
    }
    Weights pr[NR];
#pragma unroll
    for (int n = 0; n < NR; n++) pr[n] = weights(s[n]);
#pragma unroll
    for (int d0 = 0; d0 < D / 16; d0 += 4) {
      bf16x8 v[4];
#pragma unroll
      for (int d = 0; d < 4; d++) v[d] = *(const bf16x8*)(buf + Sh::v_at(16 * (d0 + d) + i, g));
#pragma unroll
      for (int e = 0; e < 2; e++)
#pragma unroll
        for (int d = 0; d < 4; d++)
#pragma unroll
          for (int n = 0; n < NR; n++)
            sum.o[n][d0 + d] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[d], e ? pr[n].lo : pr[n].hi, sum.o[n][d0 + d], 0, 0, 0);
    }
  }
  __syncthreads();  // the buffers hold outputs now
  if (idle) return;
#pragma unroll
  for (int n = 0; n < NR; n++) {
    const float l = rows_sum(sum.l[n]);
    const int r0 = row0 + 16 * n;
    if (r0 >= p.rows) break;
    if (p.splits == 1) {
      uint16_t* os = (uint16_t*)(lds + wave * OS);
      wave_fence();
      put_rows<D, D / 16>(sum.o[n], 0, l, os);
      wave_fence();
      store_rows<D>(p, b, head, r0, l, sum.m[n], os, 0, 1);
    } else {  // as they are held, 1 KB at a time
      const int64_t part = (((int64_t)b * p.a.c.heads + head) * ((p.rows + 15) / 16) + r0 / 16) * p.splits + split;
#pragma unroll
      for (int d = 0; d < D / 16; d++) *(f32x4*)(p.part_o + (part * (D / 16) + d) * 256 + 4 * lane) = sum.o[n][d];
      if (g == 0) *(f32x2*)(p.part_ml + (part * 16 + i) * 2) = f32x2{sum.m[n], l};
    }
  }
}

constexpr int MAX_PIECES = 16;  // of a request's tokens, where rows share them

// Joins the pieces of 16 rows; each wave a quarter of their dims.
template <int D>
__global__ __launch_bounds__(256) void k_attention_join_rows(AttnArgs p) {
  constexpr int ND = D / 64;
  __shared__ uint16_t os[16 * (D + 2)];
  const int lane = threadIdx.x & 63, i = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles = (p.rows + 15) / 16;
  const int64_t at = blockIdx.x;
  const int row0 = (int)(at % tiles) * 16;
  const int64_t bh = at / tiles;
  const int head = (int)(bh % p.a.c.heads), b = (int)(bh / p.a.c.heads);
  int len = p.a.lens[b];
  len = len < 0 ? 0 : (int64_t)len > p.a.max_len ? (int)p.a.max_len : len;
  // the pieces that hold tokens of the lane's row, which have all been computed
  auto pieces = [&](int row) {
    const int limit = len - p.a.Lq + 1 + (row < p.rows ? row : p.rows - 1) / p.a.group;
    return limit <= 0 ? 0 : (limit + p.chunk - 1) / p.chunk;
  };
  const int mine = pieces(row0 + i), most = pieces(row0 + 15);
  const float* ml = p.part_ml + at * p.splits * 32 + 2 * i;
  const float* po = p.part_o + (at * p.splits * (D / 16) + wave * ND) * 256 + 4 * lane;
  // sums AT pieces at a time, the next ones and all bases in flight meanwhile
  constexpr int AT = D == 256 ? 2 : 4;
  f32x4 next[AT][ND];
  auto load = [&](int s0) {
#pragma unroll
    for (int k = 0; k < AT; k++)
#pragma unroll
      for (int d = 0; d < ND; d++) {
        const int s = s0 + k < most ? s0 + k : most - 1;
        next[k][d] = *(const f32x4*)(po + ((int64_t)s * (D / 16) + d) * 256);
      }
  };
  f32x4 o[ND];
#pragma unroll
  for (int d = 0; d < ND; d++) o[d] = f32x4{0, 0, 0, 0};
  float m = -__builtin_inff(), l = 0.0f;
  if (most > 0) {
    f32x2 w[MAX_PIECES];
#pragma unroll
    for (int s = 0; s < MAX_PIECES; s++) {
      w[s] = f32x2{-__builtin_inff(), 0.0f};
      if (s < mine) w[s] = *(const f32x2*)(ml + 32 * s);
    }
    load(0);
#pragma unroll
    for (int s = 0; s < MAX_PIECES; s++) m = __builtin_fmaxf(m, w[s].x);
    const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
    for (int s0 = 0; s0 < MAX_PIECES; s0 += AT) {
      if (s0 >= most) break;
      f32x4 part[AT][ND];
#pragma unroll
      for (int k = 0; k < AT; k++)
#pragma unroll
        for (int d = 0; d < ND; d++) part[k][d] = next[k][d];
      if (s0 + AT < most) load(s0 + AT);
#pragma unroll
      for (int k = 0; k < AT; k++) {
        const float a = __builtin_amdgcn_exp2f(w[s0 + k].x - base);
        l += w[s0 + k].y * a;
#pragma unroll
        for (int d = 0; d < ND; d++)
#pragma unroll
          for (int e = 0; e < 4; e++)  // pieces that the row has no tokens in need not be numbers
            o[d][e] = s0 + k < mine ? __builtin_fmaf(part[k][d][e], a, o[d][e]) : o[d][e];
      }
    }
  }
  put_rows<D, ND>(o, wave * ND, l, os);
  __syncthreads();
  store_rows<D>(p, b, head, row0, l, m, os, wave, 4);
}

// Joins the pieces of a row.  W waves of a workgroup take a row, each of them every
// W-th piece; their sums meet in LDS.
template <int D, int W>
__global__ __launch_bounds__(256) void k_attention_join(AttnArgs p) {
  __shared__ float part[4][D + 1];
  const int64_t total = (int64_t)p.a.B * p.a.c.heads * p.rows;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t mine = (int64_t)blockIdx.x * (4 / W) + wave / W;
  const int64_t at = mine < total ? mine : total - 1;  // past the last row: that one again, not stored
  const int row = (int)(at % p.rows);
  const int64_t bh = at / p.rows;
  const int head = (int)(bh % p.a.c.heads), b = (int)(bh / p.a.c.heads);
  int len = p.a.lens[b];
  len = len < 0 ? 0 : (int64_t)len > p.a.max_len ? (int)p.a.max_len : len;
  const int qt = row / p.a.group, hq = head * p.a.group + row - qt * p.a.group;
  const int limit = len - p.a.Lq + 1 + qt;
  // the pieces that hold tokens of this row; its workgroups have computed them all
  const int n = limit <= 0 ? 0 : (limit + p.chunk - 1) / p.chunk;
  const float* mls = p.part_ml + 2 * at * p.splits;
  float m = -__builtin_inff();
  for (int s = lane; s < n; s += 64) m = __builtin_fmaxf(m, mls[2 * s]);
  m = rows_max(m);
  m = __builtin_fmaxf(m, dpp<0xB1>(m));
  m = __builtin_fmaxf(m, dpp<0x4E>(m));
  m = __builtin_fmaxf(m, dpp<0x141>(m));
  m = __builtin_fmaxf(m, dpp<0x140>(m));
  const float base = m == -__builtin_inff() ? 0.0f : m;
  float l = 0.0f, o[D / 64] = {};
#pragma unroll 4
  for (int s = wave % W; s < n; s += W) {
    const float a = __builtin_amdgcn_exp2f(mls[2 * s] - base);
    l += mls[2 * s + 1] * a;
#pragma unroll
    for (int k = 0; k < D / 64; k++) o[k] += p.part_o[(at * p.splits + s) * D + 64 * k + lane] * a;
  }
#pragma unroll
  for (int k = 0; k < D / 64; k++) part[wave][64 * k + lane] = o[k];
  if (lane == 0) part[wave][D] = l;
  __syncthreads();
  if (mine >= total) return;
  const int w0 = wave / W * W;
  l = 0.0f;
#pragma unroll
  for (int w = 0; w < W; w++) l += part[w0 + w][D];
  const int64_t tok = (int64_t)b * p.a.Lq + qt;
  for (int d = (int)threadIdx.x % (64 * W); d < D; d += 64 * W) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < W; w++) v += part[w0 + w][d];
    p.a.o[tok * p.a.ld_o + (int64_t)hq * D + d] = __builtin_bit_cast(uint16_t, (__bf16)(l == 0.0f ? 0.0f : v / l));
  }
  if (threadIdx.x % (64 * W) == 0 && p.a.lse)
    p.a.lse[tok * (p.a.c.heads * p.a.group) + hq] =
        l == 0.0f ? -__builtin_inff() : m * 0.69314718055994530942f + logf(l);
}

// Shape of the workgroups, and how the tokens are split: by sizes that the host knows,
// so a result does not depend on timing.
struct Plan {
  bool shared;  // more than 16 rows: k_attention_rows
  int nr, waves, tiles, splits, chunk;
};
// Up to 16 rows the waves of a workgroup take tokens by turns; more rows are shared
// out to them (8 requests to 4096, 8 heads of dim 128: 16 rows 22.4 us by tokens and
// 23.7 by rows; two and four tiles of 16 rows by tokens, tried with weights of one term,
// 29.4 and 35 instead of 24.0 and 27 by rows).  Workgroups are wanted twice for each
// that the chip holds at a time (two of four waves a CU, one for dim 256): 32 requests
// to 16384, dim 128, took 147 us in 4 pieces, 153 in 16 (with their join).  Few rows of up
// to 1024 tokens go to eight waves of one workgroup, without pieces and a second launch,
// and so do more tokens where requests and heads fill the chip by themselves.
// Measured, 8 heads of dim 128 (us; eight waves / pieces and their join): 1 request of
// 1000 11.3 / 10.1 and a launch more, of 2048 17.3 / 10.4; 8 to 2048 17.7 / 13.8; 16 to
// 2048 18.7 / 20.8, to 4096 30.9 / 29.1; 32 to 2048 21.4 / 29.4, to 8192 72 / 81, to 16384
// 140 / 147, but there one long request among short ones would take twice as long.
// All of it goes by max_len, which the host knows, not by the lengths, which it does not: a
// bound far above them leaves most pieces empty.
Plan plan_of(int64_t B, int64_t Lq, int heads, int group, int dim, int64_t max_len) {
  Plan r;
  const int64_t rows = Lq * group;
  r.shared = rows > 16;
  r.nr = rows > 64 && dim < 256 ? 2 : 1;
  r.tiles = r.shared ? (int)((rows + 64 * r.nr - 1) / (64 * r.nr)) : 1;
  const int64_t base = B * heads * r.tiles;
  r.waves = !r.shared && dim < 256 && max_len <= (base >= 256 ? 8192 : base >= 128 ? 2048 : 1024) ? 8 : 4;
  const int64_t unit = r.shared ? 128 : STEP * r.waves;
  const int64_t units = (max_len + unit - 1) / unit;
  int64_t splits = r.waves == 8 ? 1 : ((!r.shared && dim == 256 ? 512 : 1024) + base - 1) / base;
  if (splits > (units + 1) / 2) splits = (units + 1) / 2;  // at least two steps a wave
  if (r.shared && splits > MAX_PIECES) splits = MAX_PIECES;  // joining them costs a row's outputs each
  if (splits < 1) splits = 1;
  int64_t per = (units + splits - 1) / splits;
  if (per < 1) per = 1;
  r.chunk = (int)(per * unit);
  r.splits = (int)((units + per - 1) / per);
  if (r.splits < 1) r.splits = 1;
  return r;
}

template <int D, int F>
hipError_t attention_by_rows(const AttnArgs& p, const Plan& r, hipStream_t st) {
  const unsigned bh = (unsigned)(p.a.B * p.a.c.heads);
  const dim3 b(64 * r.waves), b4(256);
  if (r.shared) {
    const dim3 g((unsigned)r.splits, bh, (unsigned)r.tiles);
    if (r.nr == 1) hipLaunchKernelGGL((k_attention_rows<D, F, 1>), g, b, 0, st, p);
    if constexpr (D < 256)
      if (r.nr == 2) hipLaunchKernelGGL((k_attention_rows<D, F, 2>), g, b, 0, st, p);
    if (r.splits > 1)
      hipLaunchKernelGGL(k_attention_join_rows<D>, dim3(bh * (unsigned)((p.rows + 15) / 16)), b4, 0, st, p);
    return hipGetLastError();
  }
  const dim3 g((unsigned)r.splits, bh);
  if constexpr (D == 256) {
    hipLaunchKernelGGL((k_attention<D, F, 4, 1>), g, b, 0, st, p);
  } else {
    if (r.waves == 8) hipLaunchKernelGGL((k_attention<D, F, 8, 2>), g, b, 0, st, p);
    else hipLaunchKernelGGL((k_attention<D, F, 4, 2>), g, b, 0, st, p);
  }
  if (r.splits > 1) {  // 8192 rows: 12 us by four waves each, 6 by one; 32 rows of 64 pieces: 5 us and 20
    const unsigned n = bh * (unsigned)p.rows;
    if (n >= 2048) hipLaunchKernelGGL((k_attention_join<D, 1>), dim3((n + 3) / 4), b4, 0, st, p);
    else hipLaunchKernelGGL((k_attention_join<D, 4>), dim3(n), b4, 0, st, p);
  }
  return hipGetLastError();
}

template <int D>
hipError_t attention_by_fmt(const AttnArgs& p, const Plan& r, hipStream_t st) {
  return p.a.c.fmt == E4M3 ? attention_by_rows<D, E4M3>(p, r, st) : attention_by_rows<D, E5M2>(p, r, st);
}

}  // namespace

hipError_t launch_cache_write(const CacheWriteArgs& a, hipStream_t st) {
  const int shift = a.c.dim == 64 ? 3 : a.c.dim == 128 ? 4 : 5, per = a.c.heads << shift;
  const int tpw = per >= 256 ? 1 : 256 / per;
  const dim3 g = grid_of((a.tokens + tpw - 1) / tpw), b(256);
  if (a.src == SRC_BF16) {
    if (a.c.fmt == E4M3) hipLaunchKernelGGL((k_cache_write<SRC_BF16, E4M3>), g, b, 0, st, a, shift, tpw);
    else hipLaunchKernelGGL((k_cache_write<SRC_BF16, E5M2>), g, b, 0, st, a, shift, tpw);
  } else {
    if (a.c.fmt == E4M3) hipLaunchKernelGGL((k_cache_write<SRC_F32, E4M3>), g, b, 0, st, a, shift, tpw);
    else hipLaunchKernelGGL((k_cache_write<SRC_F32, E5M2>), g, b, 0, st, a, shift, tpw);
  }
  return hipGetLastError();
}

int64_t attention_workspace(int64_t B, int64_t Lq, int heads, int group, int dim, int64_t max_len) {
  const Plan r = plan_of(B, Lq, heads, group, dim, max_len);
  const int64_t rows = r.shared ? (Lq * group + 15) / 16 * 16 : Lq * group;  // whole tiles
  return r.splits == 1 ? 0 : B * heads * rows * r.splits * (dim + 2) * 4;
}

hipError_t launch_attention(const AttentionArgs& a, hipStream_t st) {
  const Plan r = plan_of(a.B, a.Lq, a.c.heads, a.group, a.c.dim, a.max_len);
  AttnArgs p;
  p.a = a;
  p.rows = a.Lq * a.group;
  p.splits = r.splits;
  p.chunk = r.chunk;
  p.page16 = (uint32_t)a.c.page / 16;
  p.magic = p.shift = 0;
  if (p.page16 > 1) {
    while ((2u << p.shift) < p.page16) p.shift++;
    p.magic = (uint32_t)(((1ull << (28 + p.shift)) + p.page16 - 1) / p.page16 << 4);
  }
  p.part_o = a.work;
  const int64_t rows = r.shared ? (p.rows + 15) / 16 * 16 : p.rows;
  p.part_ml = a.work + (int64_t)a.B * a.c.heads * rows * r.splits * a.c.dim;
  switch (a.c.dim) {
    case 64: return attention_by_fmt<64>(p, r, st);
    case 128: return attention_by_fmt<128>(p, r, st);
    default: return attention_by_fmt<256>(p, r, st);
  }
}

}  // namespace mx
