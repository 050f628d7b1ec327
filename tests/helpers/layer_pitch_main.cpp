// Host-only driver of the decoder-layer entry points' pitches (mx_layer_api.cpp), built with
// AddressSanitizer and UndefinedBehaviorSanitizer by tests/test_layer_pitches.py: a pitch
// whose bytes pass 64 bits is refused, that of an absent matrix is not looked at.
#include <cstdio>
#include <cstring>

#include "mx.h"
#include "mx_layer.h"

namespace mx {
static int calls = 0;
static NormArgs norm;
static NormGradArgs grad;
static CacheWriteArgs cwrite;
static AttentionArgs att;
hipError_t launch_norm_quant(const NormArgs& a, hipStream_t) { calls++; norm = a; return hipSuccess; }
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t) { calls++; grad = a; return hipSuccess; }
int64_t norm_grad_partials(int64_t, int64_t, int) { return 1; }
hipError_t launch_gemv(const GemvArgs&, hipStream_t) { calls++; return hipSuccess; }
hipError_t launch_cache_write(const CacheWriteArgs& a, hipStream_t) { calls++; cwrite = a; return hipSuccess; }
int64_t attention_workspace(int64_t, int64_t, int, int, int, int64_t) { return 0; }
hipError_t launch_attention(const AttentionArgs& a, hipStream_t) { calls++; att = a; return hipSuccess; }
}  // namespace mx

static int fails = 0;
#define CHECK(cond)                                                        \
  do {                                                                     \
    if (!(cond)) {                                                         \
      std::fprintf(stderr, "check failed line %d: %s\n", __LINE__, #cond); \
      fails++;                                                             \
    }                                                                      \
  } while (0)

int main() {
  alignas(16) static uint8_t buf[64];
  void* P = buf;
  float* F = (float*)buf;
  const int32_t* I = (const int32_t*)buf;
  mx_cache c;
  std::memset(&c, 0, sizeof c);
  c.k_q = c.v_q = P;
  c.k_s = c.v_s = buf;
  c.pages = 2;
  c.heads = 1;
  c.page = 16;
  c.dim = 64;
  const int64_t limit = (int64_t)1 << 40;
  for (int64_t big : {limit + 8, (int64_t)1 << 60, (int64_t)1 << 61, (int64_t)1 << 62, INT64_MAX - 63}) {
    for (int src = 0; src < 2; src++) {
      auto norm = [&](int64_t x, int64_t r, int64_t h, int64_t y) {
        return mx_rmsnorm_quantize(P, x, P, r, P, 2, 64, src, 0, 0.0f, P, h, P, y, P, buf, F, nullptr);
      };
      CHECK(norm(64, 64, 64, 64) == MX_OK);
      CHECK(norm(big, 64, 64, 64) == MX_ERR_UNSUPPORTED && norm(64, big, 64, 64) == MX_ERR_UNSUPPORTED);
      CHECK(norm(64, 64, big, 64) == MX_ERR_UNSUPPORTED && norm(64, 64, 64, big) == MX_ERR_UNSUPPORTED);
      auto grad = [&](int64_t dy, int64_t h, int64_t dh, int64_t dx) {
        return mx_rmsnorm_backward(P, dy, P, h, P, F, P, dh, 2, 64, src, P, dx, F, nullptr, 0, nullptr);
      };
      CHECK(grad(64, 64, 64, 64) == MX_OK);
      CHECK(grad(big, 64, 64, 64) == MX_ERR_UNSUPPORTED && grad(64, big, 64, 64) == MX_ERR_UNSUPPORTED);
      CHECK(grad(64, 64, big, 64) == MX_ERR_UNSUPPORTED && grad(64, 64, 64, big) == MX_ERR_UNSUPPORTED);
      auto write = [&](int64_t ld_k, int64_t hs_k, int64_t ld_v, int64_t hs_v) {
        return mx_cache_write(&c, P, ld_k, hs_k, P, ld_v, hs_v, src, 2, (const int64_t*)P, nullptr);
      };
      CHECK(write(64, 64, 64, 64) == MX_OK);
      CHECK(write(big, 64, 64, 64) == MX_ERR_UNSUPPORTED && write(64, big, 64, 64) == MX_ERR_UNSUPPORTED);
      CHECK(write(64, 64, big, 64) == MX_ERR_UNSUPPORTED && write(64, 64, 64, big) == MX_ERR_UNSUPPORTED);
      // absent matrices, and rows that are not there
      CHECK(mx_rmsnorm_quantize(P, 64, nullptr, big, P, 2, 64, src, 0, 0.0f, nullptr, big, nullptr, big, P, buf, F,
                                nullptr) == MX_OK);
      CHECK(mx::norm.ld_r == 0 && mx::norm.ld_h == 0 && mx::norm.ld_y == 0);
      CHECK(mx_rmsnorm_backward(P, 64, P, 64, P, F, nullptr, big, 2, 64, src, P, 64, F, nullptr, 0, nullptr) == MX_OK);
      CHECK(mx::grad.ld_dh == 0);
      CHECK(mx_rmsnorm_backward(nullptr, big, nullptr, big, nullptr, nullptr, nullptr, big, 0, 64, src, nullptr, big, F,
                                nullptr, 0, nullptr) == MX_OK);
    }
    auto att = [&](int64_t q, int64_t table, int64_t o) {
      return mx_attention(&c, P, q, I, table, I, 2, 1, 1, 1.0f, 16, (uint16_t*)P, o, F, nullptr, 0, nullptr);
    };
    CHECK(att(64, 1, 64) == MX_OK);
    CHECK(att(big, 1, 64) == MX_ERR_UNSUPPORTED && att(64, big, 64) == MX_ERR_UNSUPPORTED &&
          att(64, 1, big) == MX_ERR_UNSUPPORTED);
  }
  if (fails) return 1;
  std::printf("pitches: %d launcher calls, all checks passed\n", mx::calls);
  return 0;
}
