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
// share a workgroup.
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
  const int64_t tok = (int64_t)blockIdx.x * tokens_per_wg + sub;
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
// Rows of a key/value head are its (query token, query head) pairs; a workgroup
// takes NR tiles of 16 of them and one piece of the request's tokens, each wave 32
// tokens at a time.  Both products run on 16x16x32 bf16 matrix instructions, to
// which an element times its scale is exact:
//   S^T = K Q^T   lane (l % 16, g = l / 16) takes dims g D/4 .. of token l % 16 and
//                 feeds dims 8 j .. of them to instruction j, as the lane of Q does;
//                 it gets its row's scores of tokens 4 g .. 4 g + 3
//   O^T = V^T P^T those 8 scores (two groups of 16 tokens) are the lane's 8 of the
//                 32 of a sum over tokens as they are; the lane takes dims
//                 (l % 16) D/16 .. of the same 8 tokens and transposes 2 x 2
// so P stays in registers.  P is rounded to bf16 (up to 2^-8 of itself, like the
// output's own rounding; its sum l is of the unrounded p); scores, maxima, sums and O
// stay in fp32.
//
// Bound for a few rows: HBM, 2 (D + D / 32) bytes a token and head.  Each wave loads
// its 32 tokens in whole 1 KB runs and reads them again from its own piece of LDS:
// with loads in the operands' order (16 bytes of a token 32 bytes apart, scales byte
// by byte) 32 requests to 16384 took 165 us, 136 us now (4.9 TB/s).  The next 32
// tokens are in flight meanwhile.
struct u64x2 { uint2 lo, hi; };

constexpr int STEP = 32;  // tokens a wave takes at a time

struct AttnArgs {
  AttentionArgs a;
  int rows;              // Lq * group
  int splits;
  int chunk;             // tokens of a piece, a multiple of what its waves take at a time
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

// Where tokens 16 u .. of a request lie: row (page, head, place) of the cache.
// A page that is not one of the cache's holds no tokens.
__device__ __forceinline__ bool locate(const AttnArgs& p, const int32_t* table, int head, int tok, int64_t& row) {
  const uint32_t i16 = (uint32_t)tok >> 4;
  const uint32_t idx = p.page16 == 1 ? i16 : __umulhi(i16, p.magic);
  const int pg = table[idx];
  row = ((int64_t)pg * p.a.c.heads + head) * p.a.c.page + (int)(i16 - idx * p.page16) * 16;
  return (uint32_t)pg < (uint32_t)p.a.c.pages;
}

template <int D>
__device__ __forceinline__ uint32_t load_step(const AttnArgs& p, const int32_t* table, int head, int t0, int end,
                                              Raw<D>& x) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t there = 0;
  int64_t row[2];
#pragma unroll
  for (int u = 0; u < 2; u++) {
    bool ok = t0 + 16 * u < end;
    if (ok) ok = locate(p, table, head, t0 + 16 * u, row[u]);
    if (!ok) row[u] = 0;  // any row of the cache: what it holds is masked
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

// One step of 32 staged tokens.  `cut`: some row does not see all of them, or some
// are not there.  limit[n] is the number of them that the lane's row sees (less than
// 1: none, 32 or more: all).  `odd`: values may not be finite and rows see different
// tokens.
template <int D, int F, int NR>
__device__ __forceinline__ void take_step(uint8_t* lds, const bf16x8 (*q)[D / 32][64], float scale2, bool cut,
                                          bool odd, uint32_t there, const int (&limit)[NR], Sums<D, NR>& sum) {
  using St = Stage<D>;
  const int i = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  f32x4 s[NR][2];
#pragma unroll
  for (int n = 0; n < NR; n++) s[n][0] = s[n][1] = f32x4{0, 0, 0, 0};
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
#pragma unroll
      for (int n = 0; n < NR; n++) {
        const bf16x8 qj = q[n][2 * c + h][threadIdx.x & 63];
#pragma unroll
        for (int u = 0; u < 2; u++) s[n][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[u], qj, s[n][u], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NR; n++)
#pragma unroll
    for (int u = 0; u < 2; u++) s[n][u] *= scale2;
  if (cut) {  // after the scaling, whose sign is the caller's
#pragma unroll
    for (int n = 0; n < NR; n++)
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const int tok = 16 * (e >> 2) + 4 * g + (e & 3);
        const bool seen = tok < limit[n] && (there >> (e >> 2) & 1);
        s[n][e >> 2][e & 3] = seen ? s[n][e >> 2][e & 3] : -__builtin_inff();
      }
  }
  bf16x8 pr[NR];
#pragma unroll
  for (int n = 0; n < NR; n++) {
    float v[8], top = -__builtin_inff();
#pragma unroll
    for (int e = 0; e < 8; e++) {
      v[e] = s[n][e >> 2][e & 3];
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
  if (odd) {
    // 0 * NaN is not 0: token by token, for the rows that see it.  p takes the
    // place of the keys.
#pragma unroll
    for (int n = 0; n < NR; n++) {
      wave_fence();
      uint16_t* ps = (uint16_t*)(lds + St::K_AT);  // [row][token]
      *(uint2*)(ps + 32 * i + 4 * g) = __builtin_bit_cast(u64x2, pr[n]).lo;
      *(uint2*)(ps + 32 * i + 16 + 4 * g) = __builtin_bit_cast(u64x2, pr[n]).hi;
      wave_fence();
      for (int tok = 0; tok < STEP; tok++) {
        if (tok >= limit[n]) continue;
        const float pt = __builtin_bit_cast(float, (uint32_t)ps[32 * i + tok] << 16);
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
              sum.o[n][4 * k + d][e] = __builtin_fmaf(pt, v, sum.o[n][4 * k + d][e]);
            }
          }
      }
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < D / 64; k++) {
    uint32_t w[4][4];
    v_operands<D, F>(lds, k, w);
#pragma unroll
    for (int d = 0; d < 4; d++) {
      const bf16x8 v = operand(w[d][0], w[d][1], w[d][2], w[d][3]);
#pragma unroll
      for (int n = 0; n < NR; n++)
        sum.o[n][4 * k + d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, pr[n], sum.o[n][4 * k + d], 0, 0, 0);
    }
  }
}

template <int D, int F, int NR, int WAVES, int OCC>
__global__ __launch_bounds__(64 * WAVES, OCC) void k_attention(AttnArgs p) {
  __shared__ float ml[WAVES][NR][16][2];
  // the waves' staged tokens, then their outputs
  constexpr int OS = 4 * 16 * (D + 4), PIECE = Stage<D>::BYTES > OS ? Stage<D>::BYTES : OS;
  __shared__ __align__(16) uint8_t lds[WAVES * PIECE];
  float(*os)[16][D + 4] = (float(*)[16][D + 4])lds;
  __shared__ bf16x8 q[NR][D / 32][64];  // by lane, the same for every wave
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
  Sums<D, NR> sum;
#pragma unroll
  for (int n = 0; n < NR; n++) {
    int row = row0 + 16 * n + i;
    row = row < p.rows ? row : p.rows - 1;
    const int qt = row / p.a.group, hq = head * p.a.group + row - qt * p.a.group;
    const uint16_t* src = p.a.q + ((int64_t)b * p.a.Lq + qt) * p.a.ld_q + (int64_t)hq * D + g * (D / 4);
    for (int j = wave; j < D / 32; j += WAVES) q[n][j][lane] = *(const bf16x8*)(src + 8 * j);
    sum.m[n] = -__builtin_inff();
    sum.l[n] = 0.0f;
#pragma unroll
    for (int d = 0; d < D / 16; d++) sum.o[n][d] = f32x4{0, 0, 0, 0};
  }
  __syncthreads();
  const float scale2 = p.a.scale * 1.44269504088896340736f;  // scores in units of log 2

  int t = t0 + wave * STEP;
  if (t < t1) {
    uint8_t* mine = lds + wave * Stage<D>::BYTES;
    Raw<D> x;
    uint32_t there = load_step<D>(p, table, head, t, t1, x);
    while (true) {
      const bool cut = there != 3u || t + STEP > low;
      const uint32_t here = there;
      const bool odd = __any(stage_step<D, F>(x, mine, cut, here, t1 - t)) && p.a.Lq > 1;
      wave_fence();
      const int next = t + WAVES * STEP;
      if (next < t1) there = load_step<D>(p, table, head, next, t1, x);
      int limit[NR];
#pragma unroll
      for (int n = 0; n < NR; n++) limit[n] = lim[n] - t;
      take_step<D, F, NR>(mine, q, scale2, cut, odd, here, limit, sum);
      wave_fence();
      t = next;
      if (t >= t1) break;
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

// Row tiles and waves of a workgroup, and how the tokens are split: by sizes that
// the host knows, so a result does not depend on timing.
struct Plan {
  int nr, waves, tiles, splits, chunk;
};
// More tiles share the conversion of the tokens, as far as registers go without
// spilling (dim 128: two; four ran 60 us against 38 us for 4 requests of 64 query
// tokens to 4096).  Workgroups are wanted twice for each that the chip holds at a
// time (two of four waves a CU, one for dim 256), which evens out requests of
// different lengths: 32 requests to 16384, dim 128, took 136 us in 4 pieces, 143 in
// 16.  Up to 1024 tokens of few rows eight waves of one workgroup spare the second
// launch.
Plan plan_of(int64_t B, int64_t Lq, int heads, int group, int dim, int64_t max_len) {
  Plan r;
  const int64_t rows = Lq * group;
  r.nr = rows <= 16 || dim == 256 ? 1 : rows <= 32 || dim == 128 ? 2 : 4;
  r.waves = r.nr == 1 && dim < 256 && max_len <= 1024 ? 8 : 4;
  r.tiles = (int)((rows + 16 * r.nr - 1) / (16 * r.nr));
  const int64_t unit = STEP * r.waves, base = B * heads * r.tiles, want = dim == 256 ? 512 : 1024;
  const int64_t units = (max_len + unit - 1) / unit;
  int64_t splits = r.waves == 8 ? 1 : (want + base - 1) / base;
  if (splits > (units + 1) / 2) splits = (units + 1) / 2;  // at least two steps a wave
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
  const dim3 g((unsigned)r.splits, (unsigned)r.tiles, (unsigned)(p.a.B * p.a.c.heads)), b(64 * r.waves);
  if constexpr (D == 256) {
    hipLaunchKernelGGL((k_attention<D, F, 1, 4, 1>), g, b, 0, st, p);
  } else {
    if (r.waves == 8) hipLaunchKernelGGL((k_attention<D, F, 1, 8, 2>), g, b, 0, st, p);
    else if (r.nr == 1) hipLaunchKernelGGL((k_attention<D, F, 1, 4, 2>), g, b, 0, st, p);
    else if (r.nr == 2) hipLaunchKernelGGL((k_attention<D, F, 2, 4, 2>), g, b, 0, st, p);
    if constexpr (D == 64)
      if (r.nr == 4) hipLaunchKernelGGL((k_attention<D, F, 4, 4, 2>), g, b, 0, st, p);
  }
  if (r.splits > 1) {  // 8192 rows: 12 us by four waves each, 6 by one; 32 rows of 64 pieces: 5 us and 20
    const int64_t n = (int64_t)p.a.B * p.a.c.heads * p.rows;
    if (n >= 2048) hipLaunchKernelGGL((k_attention_join<D, 1>), dim3((unsigned)((n + 3) / 4)), dim3(256), 0, st, p);
    else hipLaunchKernelGGL((k_attention_join<D, 4>), dim3((unsigned)n), dim3(256), 0, st, p);
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
  const dim3 g((unsigned)((a.tokens + tpw - 1) / tpw)), b(256);
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
