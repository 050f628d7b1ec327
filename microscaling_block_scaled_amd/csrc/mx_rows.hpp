// mx_rows.hpp -- row-wise access shared by the kernels that read rows of fp32 or
// bf16 and write packed MX rows: streaming loads and stores, 8-code stores,
// widening, and loads that read +0 past the end of a row.
#pragma once

#include "mx_convert.hpp"

namespace mx {

enum { SRC_F32 = 0, SRC_BF16 = 1 };
// ---------------------------------------------------------------------------
// streaming global accesses: every input byte is read once, and the row-wise
// output is written in whole contiguous runs, so these bypass cache residency
// (non-temporal).  The transposed output writes 24-32 byte pieces of many
// rows; those stay ordinary stores so the L2 assembles whole lines.
// ---------------------------------------------------------------------------
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
  const u32x4 v = __builtin_nontemporal_load((const u32x4*)p);
  return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ void st_stream(uint8_t* p, uint4 v) {
  __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, (u32x4*)p);
}
__device__ __forceinline__ void st_stream(uint8_t* p, uint2 v) {
  __builtin_nontemporal_store(u32x2{v.x, v.y}, (u32x2*)p);
}
__device__ __forceinline__ void st_stream(uint8_t* p, uint32_t v) {
  __builtin_nontemporal_store(v, (uint32_t*)p);
}

// 8 codes at element offset 8 * c of a packed row; non-temporal when NT (a
// writer of whole lines), else ordinary stores that the L2 can merge with the
// neighbouring pieces of the line.
template <int F, bool NT = true>
__device__ __forceinline__ void store8(uint8_t* row, int64_t c, const Pack8& o) {
  if (Fmt<F>::bits == 8) {
    if (NT) st_stream(row + 8 * c, make_uint2(o.w[0], o.w[1]));
    else *(uint2*)(row + 8 * c) = make_uint2(o.w[0], o.w[1]);
  } else if (Fmt<F>::bits == 4) {
    if (NT) st_stream(row + 4 * c, o.w[0]);
    else *(uint32_t*)(row + 4 * c) = o.w[0];
  } else {  // 6 bytes at 6c: dword + half, or half + dword, by parity
    uint8_t* p = row + 6 * c;
    if ((c & 1) == 0) {
      *(uint32_t*)p = o.w[0];
      *(uint16_t*)(p + 4) = (uint16_t)o.w[1];
    } else {
      *(uint16_t*)p = (uint16_t)o.w[0];
      *(uint32_t*)(p + 2) = (o.w[0] >> 16) | (o.w[1] << 16);
    }
  }
}

template <int SRC>
__device__ __forceinline__ void widen8(const uint32_t* raw, uint32_t v[8]) {
  if (SRC == SRC_BF16) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = raw[i] << 16;
      v[2 * i + 1] = raw[i] & 0xFFFF0000u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = raw[i];
  }
}

// `n` elements (8 or 32) of ESZ bytes at src into raw words (two bf16 or one
// fp32 per word), of which the first `valid` exist and the rest read +0: whole
// 16-byte loads when all exist, else element by element (only the short last
// block of a row or tile).
template <int ESZ, int n, bool NT>
__device__ __forceinline__ void load_elems(const uint8_t* src, int valid, uint32_t* raw) {
  constexpr int W = n * ESZ / 4;  // words
  if (valid >= n) {
#pragma unroll
    for (int j = 0; j < W / 4; j++) {
      const uint4 t = NT ? ld_stream(src + 16 * j) : *(const uint4*)(src + 16 * j);
      raw[4 * j] = t.x; raw[4 * j + 1] = t.y; raw[4 * j + 2] = t.z; raw[4 * j + 3] = t.w;
    }
  } else {
#pragma unroll
    for (int w = 0; w < W; w++) {
      if (ESZ == 4) {
        raw[w] = w < valid ? *(const uint32_t*)(src + 4 * w) : 0u;
      } else {
        const uint32_t lo = 2 * w < valid ? *(const uint16_t*)(src + 4 * w) : 0u;
        const uint32_t hi = 2 * w + 1 < valid ? *(const uint16_t*)(src + 4 * w + 2) : 0u;
        raw[w] = lo | (hi << 16);
      }
    }
  }
}

// Launches of many workgroups: one dimension of a grid holds fewer than 2^32 threads.
constexpr int GRID_BITS = 20;
inline dim3 grid_of(int64_t workgroups) {
  const int64_t most = (int64_t)1 << GRID_BITS;
  return dim3((unsigned)(workgroups < most ? workgroups : most), (unsigned)((workgroups + most - 1) / most));
}
__device__ __forceinline__ int64_t workgroup() { return ((int64_t)blockIdx.y << GRID_BITS) + blockIdx.x; }

}  // namespace mx
