// mx_layer.h -- launchers of the decoder-layer operators, shared between the
// C-ABI layer (mx_layer_api.cpp) and the kernels.  Arguments have been
// validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {

// Root-mean-square norm.  Pitches in bytes; a null r, h, y, dh is absent.
struct NormArgs {
  const void *x, *r, *w;
  int64_t ld_x, ld_r;
  int64_t rows, cols;
  int src, fmt;
  float eps;
  void *h, *y;
  int64_t ld_h, ld_y;
  uint8_t *q, *s;
  float* rstd;
};
hipError_t launch_norm_quant(const NormArgs& a, hipStream_t st);

struct NormGradArgs {
  const void *dy, *h, *w, *dh;
  const float* rstd;
  int64_t ld_dy, ld_h, ld_dh;
  int64_t rows, cols;
  int src;
  void* dx;
  int64_t ld_dx;
  float* dw;
  float* partial;  // norm_grad_partials(rows, cols, src) rows of cols floats
};
int64_t norm_grad_partials(int64_t rows, int64_t cols, int src);
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t st);

// Products of a few tokens with E2M1 weights; ld_x, ld_y in elements.
struct GemvArgs {
  const uint16_t* x;  // bf16
  int64_t ld_x;
  const uint8_t *wq, *ws;
  int64_t M, N, K;
  void* y;
  int64_t ld_y;
  bool bf16;  // y in bf16, else fp32
};
hipError_t launch_gemv(const GemvArgs& a, hipStream_t st);

// The paged 8-bit key/value cache: elements [pages][heads][page][dim], scales
// [pages][heads][page][dim / 32], E4M3 or E5M2.
struct Cache {
  uint8_t *k_q, *k_s, *v_q, *v_s;
  int64_t pages;
  int heads, page, dim, fmt;
};
// k, v: [tokens][heads][dim]; pitches in bytes.
struct CacheWriteArgs {
  Cache c;
  const void *k, *v;
  int64_t ld_k, hs_k, ld_v, hs_v;
  int64_t tokens;
  const int64_t* slots;
  int src;
};
hipError_t launch_cache_write(const CacheWriteArgs& a, hipStream_t st);

struct AttentionArgs {
  Cache c;
  const uint16_t* q;  // bf16 [B * Lq][heads * group][dim], ld_q elements between rows
  int64_t ld_q;
  const int32_t* table;  // [B][ld_table] page of each piece of a request
  int64_t ld_table;
  const int32_t* lens;
  int B, Lq, group;
  float scale;
  int64_t max_len;
  uint16_t* o;  // bf16, ld_o elements between rows
  int64_t ld_o;
  float* lse;  // [B * Lq][heads * group] or null
  float* work;
};
// Bytes of `work` (0 where the keys of a request are not split).
int64_t attention_workspace(int64_t B, int64_t Lq, int heads, int group, int dim, int64_t max_len);
hipError_t launch_attention(const AttentionArgs& a, hipStream_t st);

}  // namespace mx
