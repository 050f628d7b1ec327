// mx_norm.hip -- root-mean-square norm with the residual's addition and MX
// output, and its gradient, for gfx950.
//
//   h = RN(x + r)          (r absent: h = x), rounded to the source type
//   rstd = 1 / sqrt(mean(h^2) + eps)
//   y = h * rstd * w       in fp32
//   (q, s) = Algorithm 1 of "Microscaling Data Formats for Deep Learning"
//            (summary section 3) on y: row blocks of 32, round to nearest even
//
// and for the gradient dy of y, with xhat = h * rstd and g = dy * w:
//   dx = rstd * (g - xhat * mean(g * xhat)) + dh      (dh: the gradient of h)
//   dw = sum over rows of dy * xhat
//
// Bound: HBM; for a few rows the launch and the latency of two passes of a wave over
// its registers.  A row is read once and stays in registers between the sum over the
// row and the output.  A lane holds chunks of 8 consecutive elements, so the four lanes
// of a quad hold one MX block and its maximum takes two DPP exchanges.  A row goes to
// as many waves as give each lane one chunk (one for up to 512 elements, eight from
// 2049 on), and to more chunks a lane only beyond 4096 elements.
// Measured: 16384 x 4096 bf16 with a residual, 472 MB: 85 us (5.6 TB/s; a copy of
// 1 GiB runs at 5.2); one row of 4096: 2.7 us.  8192 x 4096 with a residual (us; bf16 /
// fp32): E4M3 42.7 / 84, E2M1 43.0 / 85, INT8 45 / 88, E2M3 and E3M2, whose stores are
// of 4 and 2 bytes, 53 and 56 / 89 and 91.  The gradient of 8192 x 4096 with dh, 268 MB:
// 45 us and 4.7 us for the sum of the partial sums; fp32, 537 MB: 97 us and 4.8.
#include "mx_layer.h"
#include "mx_rows.hpp"
#include "mx_wave.hpp"

#pragma clang fp contract(off)

namespace mx {

namespace {

constexpr int WG = 512;  // threads per workgroup

// 8 elements at src + 8 c: whole chunks by 16-byte loads, a chunk past the
// row's end as zeros.  The row's last, partly filled chunk is left to
// load_tail, so that no load waits for another's branch.
template <int ESZ>
__device__ __forceinline__ void load_chunk(const uint8_t* row, int c, int cols, uint32_t raw[2 * ESZ]) {
#pragma unroll
  for (int i = 0; i < 2 * ESZ; i++) raw[i] = 0;
  if (8 * c + 8 <= cols) {
    const uint8_t* src = row + (int64_t)c * 8 * ESZ;
#pragma unroll
    for (int j = 0; j < ESZ / 2; j++) {
      const uint4 t = *(const uint4*)(src + 16 * j);
      raw[4 * j] = t.x; raw[4 * j + 1] = t.y; raw[4 * j + 2] = t.z; raw[4 * j + 3] = t.w;
    }
  }
}
template <int ESZ>
__device__ __forceinline__ void load_tail(const uint8_t* row, int c, int cols, uint32_t raw[2 * ESZ]) {
  const int valid = cols - 8 * c;
  if (valid > 0 && valid < 8) load_elems<ESZ, 8, false>(row + (int64_t)c * 8 * ESZ, valid, raw);
}
// the same for stores; elements past the row's end are not written
template <int ESZ>
__device__ __forceinline__ void store_chunk(uint8_t* row, int c, int cols, const uint32_t raw[2 * ESZ]) {
  const int valid = cols - 8 * c;
  uint8_t* dst = row + (int64_t)c * 8 * ESZ;
  if (valid >= 8) {
#pragma unroll
    for (int j = 0; j < ESZ / 2; j++)
      *(uint4*)(dst + 16 * j) = make_uint4(raw[4 * j], raw[4 * j + 1], raw[4 * j + 2], raw[4 * j + 3]);
  } else if (valid > 0) {
#pragma unroll
    for (int k = 0; k < 8; k++) {
      if (k >= valid) break;
      if (ESZ == 4) *(uint32_t*)(dst + 4 * k) = raw[k & (2 * ESZ - 1)];
      else *(uint16_t*)(dst + 2 * k) = (uint16_t)(raw[k >> 1] >> (16 * (k & 1)));
    }
  }
}

template <int SRC>
__device__ __forceinline__ void as_f32(const uint32_t* raw, float v[8]) {
  uint32_t u[8];
  widen8<SRC>(raw, u);
#pragma unroll
  for (int k = 0; k < 8; k++) v[k] = __builtin_bit_cast(float, u[k]);
}
// fp32 values to the source type, round to nearest even
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
template <int SRC>
__device__ __forceinline__ void narrow8(const float v[8], uint32_t* raw) {
  if (SRC == SRC_BF16) {
#pragma unroll
    for (int i = 0; i < 4; i++)
      raw[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){v[2 * i], v[2 * i + 1]}, bf16x2));
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) raw[i] = __builtin_bit_cast(uint32_t, v[i]);
  }
}

// sum over the W waves that share a row; `red` holds W floats.  One barrier,
// and the caller alternates between two such buffers.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if (W == 1) return v;
  if ((threadIdx.x & 63) == 0) red[(threadIdx.x >> 6) & (W - 1)] = v;
  __syncthreads();
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < W; i++) v += red[i];
  return v;
}

__device__ __forceinline__ float inv_rms(float sum, int cols, float eps) {
  return 1.0f / __builtin_sqrtf(sum / (float)cols + eps);
}

// h of one chunk: x, or x + r rounded to the source type
template <int SRC>
__device__ __forceinline__ void add_residual(const uint32_t* x, const uint32_t* r, uint32_t* h) {
  float a[8], b[8];
  as_f32<SRC>(x, a);
  as_f32<SRC>(r, b);
#pragma unroll
  for (int k = 0; k < 8; k++) a[k] += b[k];
  narrow8<SRC>(a, h);
}

// y of one chunk, its codes and scale (the quad's four lanes active together)
template <int SRC, int F>
__device__ __forceinline__ void write_chunk(const NormArgs& p, int64_t row, int c, const uint32_t* hraw,
                                            const uint32_t* wraw, float rstd) {
  constexpr int ESZ = SRC == SRC_BF16 ? 2 : 4;
  const int bpr = ((int)p.cols + 31) >> 5;
  float h[8], w[8];
  as_f32<SRC>(hraw, h);
  as_f32<SRC>(wraw, w);
  uint32_t v[8], am = 0;
#pragma unroll
  for (int k = 0; k < 8; k++) {
    h[k] = h[k] * rstd * w[k];
    // past the row's end (h = w = 0): zeros also where rstd is not finite
    if (8 * c + k >= (int)p.cols) h[k] = 0.0f;
    v[k] = __builtin_bit_cast(uint32_t, h[k]);
    am = umax(am, v[k] & 0x7FFFFFFFu);
  }
  if (p.y) {
    uint32_t yraw[2 * ESZ];
    narrow8<SRC>(h, yraw);
    store_chunk<ESZ>((uint8_t*)p.y + row * p.ld_y, c, (int)p.cols, yraw);
  }
  am = umax(am, quad_xor1(am));
  am = umax(am, quad_xor2(am));
  const uint32_t code = scale_code<F>(am);
  if ((c & 3) == 0) p.s[row * bpr + (c >> 2)] = (uint8_t)code;
  uint32_t rnd[8];
  const Pack8 o = convert8<F, false>(v, code, rnd);
  store8<F, false>(p.q + row * (bpr * (4 * Fmt<F>::bits)), c, o);
}

// Rows by W waves each, NC chunks a lane.
template <int SRC, int F, int W, int NC>
__global__ __launch_bounds__(W < 8 ? 256 : WG) void k_norm_quant(NormArgs p) {
  constexpr int ESZ = SRC == SRC_BF16 ? 2 : 4;
  constexpr int T = 64 * W, RPB = W < 8 ? 4 / W : 1;
  __shared__ float red[8];
  const int t = (int)threadIdx.x & (T - 1);
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / T);
  const int64_t last = workgroup() * RPB + group;
  // past the last row: a row of no elements, for the barrier's sake
  const bool live = last < p.rows;
  const int64_t row = live ? last : 0;
  const int cols = live ? (int)p.cols : 0, nch = (cols + 31) / 32 * 4;
  const uint8_t* x = (const uint8_t*)p.x + row * p.ld_x;
  const uint8_t* r = p.r ? (const uint8_t*)p.r + row * p.ld_r : nullptr;
  uint32_t h[NC][2 * ESZ], w[NC][2 * ESZ];
#pragma unroll
  for (int i = 0; i < NC; i++) load_chunk<ESZ>(x, t + T * i, cols, h[i]);
  if (cols & 7) {
#pragma unroll
    for (int i = 0; i < NC; i++) load_tail<ESZ>(x, t + T * i, cols, h[i]);
  }
  if (r) {
    uint32_t rr[NC][2 * ESZ];
#pragma unroll
    for (int i = 0; i < NC; i++) load_chunk<ESZ>(r, t + T * i, cols, rr[i]);
    if (cols & 7) {
#pragma unroll
      for (int i = 0; i < NC; i++) load_tail<ESZ>(r, t + T * i, cols, rr[i]);
    }
#pragma unroll
    for (int i = 0; i < NC; i++) add_residual<SRC>(h[i], rr[i], h[i]);
  }
#pragma unroll
  for (int i = 0; i < NC; i++) load_chunk<ESZ>((const uint8_t*)p.w, t + T * i, cols, w[i]);
  if (cols & 7) {
#pragma unroll
    for (int i = 0; i < NC; i++) load_tail<ESZ>((const uint8_t*)p.w, t + T * i, cols, w[i]);
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; i++) {
    float v[8];
    as_f32<SRC>(h[i], v);
#pragma unroll
    for (int k = 0; k < 8; k++) sum = __builtin_fmaf(v[k], v[k], sum);
    if (p.h) store_chunk<ESZ>((uint8_t*)p.h + row * p.ld_h, t + T * i, cols, h[i]);
  }
  sum = row_sum<W>(sum, red + group * W);
  const float rstd = inv_rms(sum, cols, p.eps);
  if (t == 0 && live && p.rstd) p.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < NC; i++)
    if (t + T * i < nch) write_chunk<SRC, F>(p, row, t + T * i, h[i], w[i], rstd);
}

// Rows too wide for registers: two passes over the row, the second from the
// cache.
template <int SRC, int F>
__global__ __launch_bounds__(WG) void k_norm_quant_wide(NormArgs p) {
  constexpr int ESZ = SRC == SRC_BF16 ? 2 : 4;
  __shared__ float red[WG / 64];
  const int64_t row = workgroup();
  if (row >= p.rows) return;
  const int cols = (int)p.cols, nch = (cols + 31) / 32 * 4;
  const uint8_t* x = (const uint8_t*)p.x + row * p.ld_x;
  const uint8_t* r = p.r ? (const uint8_t*)p.r + row * p.ld_r : nullptr;
  uint8_t* ho = p.h ? (uint8_t*)p.h + row * p.ld_h : nullptr;
  auto load = [&](const uint8_t* src, int c, uint32_t* raw) {
    load_chunk<ESZ>(src, c, cols, raw);
    load_tail<ESZ>(src, c, cols, raw);
  };
  auto h_of = [&](int c, uint32_t* h) {
    load(x, c, h);
    if (r) {
      uint32_t rr[2 * ESZ];
      load(r, c, rr);
      add_residual<SRC>(h, rr, h);
    }
  };
  float sum = 0.0f;
  for (int c = threadIdx.x; c < nch; c += WG) {
    uint32_t h[2 * ESZ];
    float v[8];
    h_of(c, h);
    as_f32<SRC>(h, v);
#pragma unroll
    for (int k = 0; k < 8; k++) sum = __builtin_fmaf(v[k], v[k], sum);
    if (ho) store_chunk<ESZ>(ho, c, cols, h);
  }
  sum = row_sum<WG / 64>(sum, red);
  const float rstd = inv_rms(sum, cols, p.eps);
  if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
  for (int c = threadIdx.x; c < nch; c += WG) {
    uint32_t h[2 * ESZ], w[2 * ESZ];
    // h may be x or r: then they now hold h, which this thread wrote
    if (ho) load(ho, c, h);
    else h_of(c, h);
    load((const uint8_t*)p.w, c, w);
    write_chunk<SRC, F>(p, row, c, h, w, rstd);
  }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
// A workgroup takes rows b, b + grid, ... (eight at a time where a wave holds a
// row) and keeps its share of dw in registers; the shares of the waves meet in
// LDS in a fixed order, and each workgroup writes one row of partial sums.
template <int SRC>
__device__ __forceinline__ void grad_chunk_sums(const uint32_t* h, const uint32_t* dy, const uint32_t* w,
                                                float rstd, float& dot, float dw[8]) {
  float a[8], b[8], c[8];
  as_f32<SRC>(h, a);
  as_f32<SRC>(dy, b);
  as_f32<SRC>(w, c);
#pragma unroll
  for (int k = 0; k < 8; k++) {
    const float t = b[k] * (a[k] * rstd);  // dy * xhat
    dw[k] += t;
    dot = __builtin_fmaf(t, c[k], dot);
  }
}
template <int SRC>
__device__ __forceinline__ void grad_chunk_dx(const uint32_t* h, const uint32_t* dy, const uint32_t* w,
                                              const uint32_t* dh, float rstd, float mean, uint32_t* out) {
  float a[8], b[8], c[8], d[8];
  as_f32<SRC>(h, a);
  as_f32<SRC>(dy, b);
  as_f32<SRC>(w, c);
  as_f32<SRC>(dh, d);
#pragma unroll
  for (int k = 0; k < 8; k++) {
    const float xhat = a[k] * rstd;
    a[k] = __builtin_fmaf(rstd, b[k] * c[k] - xhat * mean, d[k]);
  }
  narrow8<SRC>(a, out);
}

template <int SRC, int W, int NC>
__global__ __launch_bounds__(WG) void k_norm_grad(NormGradArgs p) {
  constexpr int ESZ = SRC == SRC_BF16 ? 2 : 4;
  constexpr int T = 64 * W, RPB = WG / T;  // rows a workgroup takes at a time
  __shared__ float red[2][WG / 64];
  __shared__ __align__(16) float share[RPB > 1 ? 8 * T * NC : 1];
  const int t = (int)threadIdx.x & (T - 1);
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / T);
  const int cols = (int)p.cols;
  float dw[NC][8];
  uint32_t w[NC][2 * ESZ];
#pragma unroll
  for (int i = 0; i < NC; i++) {
#pragma unroll
    for (int k = 0; k < 8; k++) dw[i][k] = 0.0f;
    load_chunk<ESZ>((const uint8_t*)p.w, t + T * i, cols, w[i]);
    load_tail<ESZ>((const uint8_t*)p.w, t + T * i, cols, w[i]);
  }
  const float inv_n = 1.0f / (float)cols;
  // a row's chunks; rows past the last are zeros
  struct Row {
    uint32_t h[NC][2 * ESZ], dy[NC][2 * ESZ], dh[NC][2 * ESZ];
    float rstd;
  };
  auto load_row = [&](int64_t row, Row& x) {
    const bool live = row < p.rows;
    const int n = live ? cols : 0;
    row = live ? row : 0;
    const uint8_t* hr = (const uint8_t*)p.h + row * p.ld_h;
    const uint8_t* dyr = (const uint8_t*)p.dy + row * p.ld_dy;
    const uint8_t* dhr = (const uint8_t*)p.dh + row * p.ld_dh;
    x.rstd = live ? p.rstd[row] : 0.0f;
#pragma unroll
    for (int i = 0; i < NC; i++) {
      load_chunk<ESZ>(hr, t + T * i, n, x.h[i]);
      load_chunk<ESZ>(dyr, t + T * i, n, x.dy[i]);
      load_chunk<ESZ>(dhr, t + T * i, p.dh ? n : 0, x.dh[i]);
    }
    if (cols & 7) {
#pragma unroll
      for (int i = 0; i < NC; i++) {
        load_tail<ESZ>(hr, t + T * i, n, x.h[i]);
        load_tail<ESZ>(dyr, t + T * i, n, x.dy[i]);
        load_tail<ESZ>(dhr, t + T * i, p.dh ? n : 0, x.dh[i]);
      }
    }
  };
  Row x;
  load_row((int64_t)blockIdx.x * RPB + group, x);
  int turn = 0;
  // the same number of turns for every wave of the workgroup
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < p.rows; base += (int64_t)gridDim.x * RPB, turn ^= 1) {
    const int64_t row = base + group;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; i++) grad_chunk_sums<SRC>(x.h[i], x.dy[i], w[i], x.rstd, dot, dw[i]);
    Row ahead;
    load_row(row + (int64_t)gridDim.x * RPB, ahead);
    const float mean = row_sum<W>(dot, red[turn] + group * W) * inv_n;
    uint8_t* dxr = (uint8_t*)p.dx + row * p.ld_dx;
#pragma unroll
    for (int i = 0; i < NC; i++) {
      uint32_t o[2 * ESZ];
      grad_chunk_dx<SRC>(x.h[i], x.dy[i], w[i], x.dh[i], x.rstd, mean, o);
      store_chunk<ESZ>(dxr, t + T * i, row < p.rows ? cols : 0, o);
    }
    x = ahead;
  }
  float* out = p.partial + (int64_t)blockIdx.x * cols;
  if constexpr (RPB > 1) {  // the groups add their shares one after the other
    for (int v = 0; v < RPB; v++) {
      if (group == v) {
#pragma unroll
        for (int i = 0; i < NC; i++) {
          float* s = share + 8 * (t + T * i);
#pragma unroll
          for (int k = 0; k < 8; k++) {
            dw[i][k] += v ? s[k] : 0.0f;
            s[k] = dw[i][k];
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < cols; c += WG) out[c] = share[c];
  } else {
#pragma unroll
    for (int i = 0; i < NC; i++)
#pragma unroll
      for (int k = 0; k < 8; k++)
        if (8 * (t + T * i) + k < cols) out[8 * (t + T * i) + k] = dw[i][k];
  }
}

// Rows too wide for registers: dx by two passes over each row ...
template <int SRC>
__global__ __launch_bounds__(WG) void k_norm_grad_wide(NormGradArgs p) {
  constexpr int ESZ = SRC == SRC_BF16 ? 2 : 4;
  __shared__ float red[WG / 64];
  const int64_t row = blockIdx.x;
  const int cols = (int)p.cols, nch = (cols + 7) / 8;
  auto load = [&](const void* src, int64_t ld, int c, uint32_t* raw) {
    const uint8_t* s = (const uint8_t*)src + row * ld;
    load_chunk<ESZ>(s, c, cols, raw);
    load_tail<ESZ>(s, c, cols, raw);
  };
  const float rstd = p.rstd[row];
  float dot = 0.0f;
  for (int c = threadIdx.x; c < nch; c += WG) {
    uint32_t h[2 * ESZ], dy[2 * ESZ], w[2 * ESZ];
    float none[8] = {};
    load(p.h, p.ld_h, c, h);
    load(p.dy, p.ld_dy, c, dy);
    load(p.w, 0, c, w);
    grad_chunk_sums<SRC>(h, dy, w, rstd, dot, none);
  }
  const float mean = row_sum<WG / 64>(dot, red) * (1.0f / (float)cols);
  for (int c = threadIdx.x; c < nch; c += WG) {
    uint32_t h[2 * ESZ], dy[2 * ESZ], w[2 * ESZ], dh[2 * ESZ] = {}, o[2 * ESZ];
    load(p.h, p.ld_h, c, h);
    load(p.dy, p.ld_dy, c, dy);
    load(p.w, 0, c, w);
    if (p.dh) load(p.dh, p.ld_dh, c, dh);
    grad_chunk_dx<SRC>(h, dy, w, dh, rstd, mean, o);
    store_chunk<ESZ>((uint8_t*)p.dx + row * p.ld_dx, c, cols, o);
  }
}
// ... and dw by columns: workgroup (b, v) sums 8 * WG columns over rows
// v, v + gridDim.y, ...  It runs before k_norm_grad_wide, since dx may be dy.
template <int SRC>
__global__ __launch_bounds__(WG) void k_norm_dw_wide(NormGradArgs p) {
  constexpr int ESZ = SRC == SRC_BF16 ? 2 : 4;
  const int cols = (int)p.cols, c = blockIdx.x * WG + threadIdx.x;
  float dw[8] = {};
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    uint32_t h[2 * ESZ], dy[2 * ESZ];
    const uint8_t *hr = (const uint8_t*)p.h + row * p.ld_h, *dyr = (const uint8_t*)p.dy + row * p.ld_dy;
    load_chunk<ESZ>(hr, c, cols, h);
    load_chunk<ESZ>(dyr, c, cols, dy);
    load_tail<ESZ>(hr, c, cols, h);
    load_tail<ESZ>(dyr, c, cols, dy);
    float none = 0.0f;
    grad_chunk_sums<SRC>(h, dy, h, p.rstd[row], none, dw);
  }
  float* out = p.partial + (int64_t)blockIdx.y * cols;
#pragma unroll
  for (int k = 0; k < 8; k++)
    if (8 * c + k < cols) out[8 * c + k] = dw[k];
}

// dw[c] = sum of the n partial rows, 16 interleaved sums of a column joined in
// a fixed order.
__global__ __launch_bounds__(1024) void k_sum_partials(const float* __restrict__ partial, int n, int64_t cols,
                                                       float* __restrict__ dw) {
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, v = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int i = v; i < n; i += 16) s += partial[(int64_t)i * cols + c];
  }
  part[v][lane] = s;
  __syncthreads();
  if (v == 0 && c < cols) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i++) s += part[i][lane];
    dw[c] = s;
  }
}

constexpr int64_t kMaxCols = 16384;  // 8 waves x 64 lanes x 4 chunks of 8
// the gradient kernel's row in registers: h, dy, dh, the next row's, w and dw
constexpr int64_t grad_max_cols(int src) { return src == SRC_BF16 ? 16384 : 8192; }

// Waves a row.  Measured (us; as here / half the waves with two chunks a lane / eight
// waves): 16384 x 1024 22.9 / 23.7 / 38.1, 8192 x 2048 23.3 / 24.0 / 25.1,
// 8192 x 4096 42.3 / 47.2 / 42.3; 16384 x 512 14.4 and by eight waves 35.0.
template <int SRC, int F>
hipError_t norm_launch(const NormArgs& a, hipStream_t st) {
  const dim3 b(a.cols <= 2048 ? 256 : WG);
  auto grid = [&](int per) { return grid_of((a.rows + per - 1) / per); };
  if (a.cols <= 512) hipLaunchKernelGGL((k_norm_quant<SRC, F, 1, 1>), grid(4), b, 0, st, a);
  else if (a.cols <= 1024) hipLaunchKernelGGL((k_norm_quant<SRC, F, 2, 1>), grid(2), b, 0, st, a);
  else if (a.cols <= 2048) hipLaunchKernelGGL((k_norm_quant<SRC, F, 4, 1>), grid(1), b, 0, st, a);
  else if (a.cols <= 4096) hipLaunchKernelGGL((k_norm_quant<SRC, F, 8, 1>), grid(1), b, 0, st, a);
  else if (a.cols <= 8192) hipLaunchKernelGGL((k_norm_quant<SRC, F, 8, 2>), grid(1), b, 0, st, a);
  else if (a.cols <= kMaxCols) hipLaunchKernelGGL((k_norm_quant<SRC, F, 8, 4>), grid(1), b, 0, st, a);
  else hipLaunchKernelGGL((k_norm_quant_wide<SRC, F>), grid(1), b, 0, st, a);
  return hipGetLastError();
}

template <int SRC>
hipError_t norm_by_fmt(const NormArgs& a, hipStream_t st) {
  switch (a.fmt) {
    case E4M3: return norm_launch<SRC, E4M3>(a, st);
    case E5M2: return norm_launch<SRC, E5M2>(a, st);
    case E2M3: return norm_launch<SRC, E2M3>(a, st);
    case E3M2: return norm_launch<SRC, E3M2>(a, st);
    case E2M1: return norm_launch<SRC, E2M1>(a, st);
    default: return norm_launch<SRC, INT8>(a, st);
  }
}

// Waves that share a row in the gradient kernel: a chunk a lane where eight waves
// suffice.  Measured (us; as here / half the waves with two chunks / eight waves):
// 16384 x 1024 24.1 / 24.4 / 53.1, 8192 x 2048 23.7 / 24.1 / 32.0,
// 8192 x 4096 44.5 / 44.5 / 44.4.
int grad_waves(int64_t cols) { return cols <= 512 ? 1 : cols <= 1024 ? 2 : cols <= 2048 ? 4 : 8; }

template <int SRC>
hipError_t grad_launch(NormGradArgs a, hipStream_t st) {
  const int64_t n = norm_grad_partials(a.rows, a.cols, SRC);
  const dim3 g((unsigned)n), b(WG);
  if (n == 1) a.partial = a.dw;
  if (a.rows == 0) {  // dw is a sum of nothing
  } else if (a.cols > grad_max_cols(SRC)) {
    const dim3 gc((unsigned)((a.cols + 8 * WG - 1) / (8 * WG)), (unsigned)n);
    hipLaunchKernelGGL(k_norm_dw_wide<SRC>, gc, b, 0, st, a);
    hipLaunchKernelGGL(k_norm_grad_wide<SRC>, dim3((unsigned)a.rows), b, 0, st, a);
  } else {
    if (a.cols <= 512) hipLaunchKernelGGL((k_norm_grad<SRC, 1, 1>), g, b, 0, st, a);
    else if (a.cols <= 1024) hipLaunchKernelGGL((k_norm_grad<SRC, 2, 1>), g, b, 0, st, a);
    else if (a.cols <= 2048) hipLaunchKernelGGL((k_norm_grad<SRC, 4, 1>), g, b, 0, st, a);
    else if (a.cols <= 4096) hipLaunchKernelGGL((k_norm_grad<SRC, 8, 1>), g, b, 0, st, a);
    else if (a.cols <= 8192) hipLaunchKernelGGL((k_norm_grad<SRC, 8, 2>), g, b, 0, st, a);
    else if constexpr (SRC == SRC_BF16) hipLaunchKernelGGL((k_norm_grad<SRC, 8, 4>), g, b, 0, st, a);
  }
  if (n != 1)  // a single workgroup's partial sums are dw
    hipLaunchKernelGGL(k_sum_partials, dim3((unsigned)((a.cols + 63) / 64)), dim3(1024), 0, st,
                       (const float*)a.partial, (int)n, a.cols, a.dw);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_quant(const NormArgs& a, hipStream_t st) {
  return a.src == SRC_BF16 ? norm_by_fmt<SRC_BF16>(a, st) : norm_by_fmt<SRC_F32>(a, st);
}

// Workgroups, and so rows of partial sums of dw: one a CU (8192 x 4096, both kernels:
// 50.6 us with 256; with 128, 512 and 1024 it took longer, by the loads in flight or by
// the partial sums).
int64_t norm_grad_partials(int64_t rows, int64_t cols, int src) {
  if (cols > grad_max_cols(src)) return rows < 64 ? rows : 64;
  const int64_t per = (WG / 64) / grad_waves(cols), n = (rows + per - 1) / per;
  return n < 256 ? n : 256;
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t st) {
  return a.src == SRC_BF16 ? grad_launch<SRC_BF16>(a, st) : grad_launch<SRC_F32>(a, st);
}

}  // namespace mx
