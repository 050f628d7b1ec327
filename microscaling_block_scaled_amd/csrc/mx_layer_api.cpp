// mx_layer_api.cpp -- the C-ABI entry points of the decoder-layer operators
// declared in include/mx.h: norm, few-token products, key/value cache and
// attention.  Every argument is checked on the host before anything is
// launched.  No exception leaves this file.
#include "../../include/mx.h"

#include <hip/hip_runtime.h>

#include "mx_layer.h"

namespace {

bool fmt_ok(int32_t f) { return f >= MX_E4M3 && f <= MX_INT8; }
bool src_ok(int32_t s) { return s == MX_SRC_F32 || s == MX_SRC_BF16; }
bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ERR_HIP; }
int64_t esz_of(int32_t src) { return src == MX_SRC_F32 ? 4 : 2; }

// Elements between rows, heads or requests: no memory has them further apart, and their
// bytes stay far below 2^63.
constexpr int64_t kMaxPitch = (int64_t)1 << 40;

// A row-major matrix that may be absent: its pitch covers a row, its rows start
// on 16 bytes.
int check_rows(const void* p, int64_t ld, int64_t cols, int64_t esz) {
  if (!p) return MX_OK;
  if (ld < cols) return MX_ERR_SHAPE;
  if (ld > kMaxPitch) return MX_ERR_UNSUPPORTED;
  if (!aligned(p, 16) || (ld * esz) % 16) return MX_ERR_ALIGN;
  return MX_OK;
}
// Bytes between its rows; an absent matrix has none.
int64_t pitch_of(const void* p, int64_t ld, int64_t esz) { return p ? ld * esz : 0; }

constexpr int64_t kMaxRows = (int64_t)1 << 31;
constexpr int64_t kMaxNormCols = (int64_t)1 << 24;
constexpr int64_t kMaxGemvRows = (int64_t)1 << 26;  // of W: 32 threads a row, fewer than 2^32 in a launch

int check_cache(const mx_cache* c) {
  if (!c || !fmt_ok(c->fmt) || c->pages < 0 || c->heads < 0 || c->page <= 0 || c->dim <= 0) return MX_ERR_ARG;
  if (c->fmt != MX_E4M3 && c->fmt != MX_E5M2) return MX_ERR_UNSUPPORTED;
  if (c->dim != 64 && c->dim != 128 && c->dim != 256) return MX_ERR_UNSUPPORTED;
  if (c->page % 16 || c->page > 65536 || c->heads > 65535 || c->pages >= kMaxRows) return MX_ERR_UNSUPPORTED;
  if (c->pages > 0 && c->heads > 0) {
    if (!c->k_q || !c->k_s || !c->v_q || !c->v_s) return MX_ERR_ARG;
    if (!aligned(c->k_q, 16) || !aligned(c->k_s, 16) || !aligned(c->v_q, 16) || !aligned(c->v_s, 16))
      return MX_ERR_ALIGN;
  }
  return MX_OK;
}

mx::Cache cache_of(const mx_cache* c) {
  mx::Cache r;
  r.k_q = (uint8_t*)c->k_q;
  r.k_s = c->k_s;
  r.v_q = (uint8_t*)c->v_q;
  r.v_s = c->v_s;
  r.pages = c->pages;
  r.heads = c->heads;
  r.page = c->page;
  r.dim = c->dim;
  r.fmt = c->fmt;
  return r;
}

int gemv(const void* x, int64_t ld_x, const void* w_q, const uint8_t* w_s, int32_t w_fmt, int64_t M, int64_t N,
         int64_t K, void* y, int64_t ld_y, bool bf16, mx_stream_t stream) {
  if (!fmt_ok(w_fmt)) return MX_ERR_ARG;
  if (w_fmt != MX_E2M1) return MX_ERR_UNSUPPORTED;
  if (M < 0 || N < 0 || K < 0) return MX_ERR_ARG;
  if (ld_x < K || ld_y < N) return MX_ERR_SHAPE;
  if (M == 0 || N == 0) return MX_OK;
  if (!y || (K > 0 && (!x || !w_q || !w_s))) return MX_ERR_ARG;
  if (!aligned(x, 2) || !aligned(w_q, 16) || !aligned(y, bf16 ? 2 : 4)) return MX_ERR_ALIGN;
  if (M > (int64_t)32 * 65535 || N > kMaxGemvRows || K >= kMaxRows) return MX_ERR_UNSUPPORTED;
  mx::GemvArgs a;
  a.x = (const uint16_t*)x;
  a.ld_x = ld_x;
  a.wq = (const uint8_t*)w_q;
  a.ws = w_s;
  a.M = M;
  a.N = N;
  a.K = K;
  a.y = y;
  a.ld_y = ld_y;
  a.bf16 = bf16;
  return hip_status(mx::launch_gemv(a, (hipStream_t)stream));
}

// Sizes of an attention call; MX_OK where a plan exists for them.
int check_attention(int64_t B, int64_t Lq, int64_t heads_q, int64_t heads, int64_t dim, int64_t max_len) {
  if (B < 0 || Lq < 0 || heads_q < 0 || heads < 0 || max_len < 0) return MX_ERR_ARG;
  if (dim != 64 && dim != 128 && dim != 256) return MX_ERR_UNSUPPORTED;
  if (heads == 0 ? heads_q != 0 : heads_q % heads != 0) return MX_ERR_SHAPE;
  if (B > 65535 || heads > 65535 || B * heads > 65535 || heads_q > 65535 || Lq > ((int64_t)1 << 30) ||
      max_len > ((int64_t)1 << 30))
    return MX_ERR_UNSUPPORTED;
  if (heads > 0 && Lq * (heads_q / heads) > 16 * 65535) return MX_ERR_UNSUPPORTED;
  return MX_OK;
}

}  // namespace

extern "C" {

int mx_rmsnorm_quantize(const void* x, int64_t ld_x, const void* r, int64_t ld_r, const void* w, int64_t rows,
                        int64_t cols, int32_t src, int32_t fmt, float eps, void* h, int64_t ld_h, void* y,
                        int64_t ld_y, void* q_row, uint8_t* s_row, float* rstd, mx_stream_t stream) {
  if (!src_ok(src) || !fmt_ok(fmt) || rows < 0 || cols < 0 || !(eps >= 0.0f)) return MX_ERR_ARG;
  const int64_t esz = esz_of(src);
  if (ld_x < cols) return MX_ERR_SHAPE;
  if (rows == 0 || cols == 0) return MX_OK;
  if (!x || !w || !q_row || !s_row) return MX_ERR_ARG;
  if (rows >= kMaxRows || cols > kMaxNormCols) return MX_ERR_UNSUPPORTED;
  const void* p[] = {x, r, h, y};
  const int64_t ld[] = {ld_x, ld_r, ld_h, ld_y};
  for (int i = 0; i < 4; i++)
    if (const int e = check_rows(p[i], ld[i], cols, esz)) return e;
  if (!aligned(w, 16) || !aligned(q_row, 16) || !aligned(rstd, 4)) return MX_ERR_ALIGN;
  mx::NormArgs a;
  a.x = x;
  a.r = r;
  a.w = w;
  a.ld_x = pitch_of(x, ld_x, esz);
  a.ld_r = pitch_of(r, ld_r, esz);
  a.rows = rows;
  a.cols = cols;
  a.src = src;
  a.fmt = fmt;
  a.eps = eps;
  a.h = h;
  a.y = y;
  a.ld_h = pitch_of(h, ld_h, esz);
  a.ld_y = pitch_of(y, ld_y, esz);
  a.q = (uint8_t*)q_row;
  a.s = s_row;
  a.rstd = rstd;
  return hip_status(mx::launch_norm_quant(a, (hipStream_t)stream));
}

int64_t mx_rmsnorm_backward_workspace(int64_t rows, int64_t cols, int32_t src) {
  if (!src_ok(src) || rows < 0 || cols < 0 || rows >= kMaxRows || cols > kMaxNormCols) return -1;
  const int64_t n = mx::norm_grad_partials(rows, cols, src);
  return n > 1 ? n * cols * 4 : 0;
}

int mx_rmsnorm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h, const void* w,
                        const float* rstd, const void* dh, int64_t ld_dh, int64_t rows, int64_t cols,
                        int32_t src, void* dx, int64_t ld_dx, float* dw, void* workspace,
                        int64_t workspace_bytes, mx_stream_t stream) {
  if (!src_ok(src) || rows < 0 || cols < 0) return MX_ERR_ARG;
  if (cols == 0) return MX_OK;
  if (!dw) return MX_ERR_ARG;
  if (rows >= kMaxRows || cols > kMaxNormCols) return MX_ERR_UNSUPPORTED;
  if (!aligned(dw, 4)) return MX_ERR_ALIGN;
  const int64_t esz = esz_of(src);
  if (rows > 0) {
    if (!dy || !h || !w || !rstd || !dx) return MX_ERR_ARG;
    const void* p[] = {dy, h, dh, dx};
    const int64_t ld[] = {ld_dy, ld_h, ld_dh, ld_dx};
    for (int i = 0; i < 4; i++)
      if (const int e = check_rows(p[i], ld[i], cols, esz)) return e;
    if (!aligned(w, 16) || !aligned(rstd, 4)) return MX_ERR_ALIGN;
    const int64_t need = mx_rmsnorm_backward_workspace(rows, cols, src);
    if (need > 0) {
      if (!workspace) return MX_ERR_ARG;
      if (!aligned(workspace, 16)) return MX_ERR_ALIGN;
      if (workspace_bytes < need) return MX_ERR_SHAPE;
    }
  }
  if (rows == 0) {  // there are no rows, whatever their pitches are said to be
    dy = h = dh = nullptr;
    dx = nullptr;
  }
  mx::NormGradArgs a;
  a.dy = dy;
  a.h = h;
  a.w = w;
  a.dh = dh;
  a.rstd = rstd;
  a.ld_dy = pitch_of(dy, ld_dy, esz);
  a.ld_h = pitch_of(h, ld_h, esz);
  a.ld_dh = pitch_of(dh, ld_dh, esz);
  a.rows = rows;
  a.cols = cols;
  a.src = src;
  a.dx = dx;
  a.ld_dx = pitch_of(dx, ld_dx, esz);
  a.dw = dw;
  a.partial = (float*)workspace;
  return hip_status(mx::launch_norm_grad(a, (hipStream_t)stream));
}

int mx_gemv(const void* x, int64_t ld_x, const void* w_q, const uint8_t* w_s, int32_t w_fmt, int64_t M, int64_t N,
            int64_t K, float* y, int64_t ld_y, mx_stream_t stream) {
  return gemv(x, ld_x, w_q, w_s, w_fmt, M, N, K, y, ld_y, false, stream);
}

int mx_gemv_bf16(const void* x, int64_t ld_x, const void* w_q, const uint8_t* w_s, int32_t w_fmt, int64_t M,
                 int64_t N, int64_t K, uint16_t* y, int64_t ld_y, mx_stream_t stream) {
  return gemv(x, ld_x, w_q, w_s, w_fmt, M, N, K, y, ld_y, true, stream);
}

int mx_cache_write(const mx_cache* cache, const void* k, int64_t ld_k, int64_t hs_k, const void* v, int64_t ld_v,
                   int64_t hs_v, int32_t src, int64_t tokens, const int64_t* slots, mx_stream_t stream) {
  if (const int e = check_cache(cache)) return e;
  if (!src_ok(src) || tokens < 0 || ld_k < 0 || hs_k < 0 || ld_v < 0 || hs_v < 0) return MX_ERR_ARG;
  if (tokens == 0 || cache->heads == 0 || cache->pages == 0) return MX_OK;
  if (!k || !v || !slots) return MX_ERR_ARG;
  if (tokens >= kMaxRows || ld_k > kMaxPitch || hs_k > kMaxPitch || ld_v > kMaxPitch || hs_v > kMaxPitch)
    return MX_ERR_UNSUPPORTED;
  const int64_t esz = esz_of(src);
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8) || (ld_k * esz) % 16 || (hs_k * esz) % 16 ||
      (ld_v * esz) % 16 || (hs_v * esz) % 16)
    return MX_ERR_ALIGN;
  mx::CacheWriteArgs a;
  a.c = cache_of(cache);
  a.k = k;
  a.v = v;
  a.ld_k = ld_k * esz;
  a.hs_k = hs_k * esz;
  a.ld_v = ld_v * esz;
  a.hs_v = hs_v * esz;
  a.tokens = tokens;
  a.slots = slots;
  a.src = src;
  return hip_status(mx::launch_cache_write(a, (hipStream_t)stream));
}

int64_t mx_attention_workspace(int64_t B, int64_t Lq, int64_t heads_q, int64_t heads, int64_t dim,
                               int64_t max_len) {
  if (check_attention(B, Lq, heads_q, heads, dim, max_len)) return -1;
  if (B == 0 || Lq == 0 || heads_q == 0) return 0;
  return mx::attention_workspace(B, Lq, (int)heads, (int)(heads_q / heads), (int)dim, max_len);
}

int mx_attention(const mx_cache* cache, const void* q, int64_t ld_q, const int32_t* table, int64_t ld_table,
                 const int32_t* lens, int64_t B, int64_t Lq, int64_t heads_q, float scale, int64_t max_len,
                 uint16_t* o, int64_t ld_o, float* lse, void* workspace, int64_t workspace_bytes,
                 mx_stream_t stream) {
  if (const int e = check_cache(cache)) return e;
  if (const int e = check_attention(B, Lq, heads_q, cache->heads, cache->dim, max_len)) return e;
  if (ld_q < heads_q * cache->dim || ld_o < heads_q * cache->dim) return MX_ERR_SHAPE;
  if (ld_table < 0 || (max_len + cache->page - 1) / cache->page > ld_table) return MX_ERR_SHAPE;
  if (B == 0 || Lq == 0 || heads_q == 0) return MX_OK;
  if (!q || !o || !lens || (max_len > 0 && !table)) return MX_ERR_ARG;
  if (ld_q > kMaxPitch || ld_o > kMaxPitch || ld_table > kMaxPitch) return MX_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || (ld_q * 2) % 16 || !aligned(o, 2) || !aligned(lse, 4) || !aligned(table, 4) ||
      !aligned(lens, 4))
    return MX_ERR_ALIGN;
  const int64_t need = mx_attention_workspace(B, Lq, heads_q, cache->heads, cache->dim, max_len);
  if (need > 0) {
    if (!workspace) return MX_ERR_ARG;
    if (!aligned(workspace, 16)) return MX_ERR_ALIGN;
    if (workspace_bytes < need) return MX_ERR_SHAPE;
  }
  if (cache->pages == 0) max_len = 0;  // there are no tokens, and no memory that stands in for absent ones
  mx::AttentionArgs a;
  a.c = cache_of(cache);
  a.q = (const uint16_t*)q;
  a.ld_q = ld_q;
  a.table = table;
  a.ld_table = ld_table;
  a.lens = lens;
  a.B = (int)B;
  a.Lq = (int)Lq;
  a.group = (int)(heads_q / cache->heads);
  a.scale = scale;
  a.max_len = max_len;
  a.o = o;
  a.ld_o = ld_o;
  a.lse = lse;
  a.work = (float*)workspace;
  return hip_status(mx::launch_attention(a, (hipStream_t)stream));
}

}  // extern "C"
