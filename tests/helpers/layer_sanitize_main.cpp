// Host-only driver of the decoder-layer entry points (mx_layer_api.cpp), built with
// AddressSanitizer and UndefinedBehaviorSanitizer by tests/test_layer_sanitizers.py.
// The kernel launchers are replaced by stubs that record what validation hands them.
#include <cmath>
#include <cstdio>
#include <cstring>

#include "mx.h"
#include "mx_layer.h"

namespace mx {
static int calls = 0;
static NormArgs norm;
static NormGradArgs grad;
static GemvArgs gemv;
static CacheWriteArgs cwrite;
static AttentionArgs att;
hipError_t launch_norm_quant(const NormArgs& a, hipStream_t) { calls++; norm = a; return hipSuccess; }
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t) { calls++; grad = a; return hipSuccess; }
int64_t norm_grad_partials(int64_t rows, int64_t, int) { return rows < 256 ? rows : 256; }
hipError_t launch_gemv(const GemvArgs& a, hipStream_t) { calls++; gemv = a; return hipSuccess; }
hipError_t launch_cache_write(const CacheWriteArgs& a, hipStream_t) { calls++; cwrite = a; return hipSuccess; }
int64_t attention_workspace(int64_t, int64_t, int, int, int, int64_t max_len) { return max_len > 1024 ? 4096 : 0; }
hipError_t launch_attention(const AttentionArgs& a, hipStream_t) { calls++; att = a; return hipErrorUnknown; }
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
  alignas(16) static uint8_t buf[1 << 12];
  void* P = buf;
  float* F = (float*)buf;
  const int64_t big = (int64_t)1 << 62;
  for (int src = 0; src < 2; src++)
    for (int fmt = 0; fmt < 6; fmt++)
      for (int64_t cols : {1, 31, 32, 4100}) {
        const int64_t ld = (cols + 7) / 8 * 8;
        CHECK(mx_rmsnorm_quantize(P, ld, P, ld, P, 3, cols, src, fmt, 0.0f, P, ld, nullptr, 0, P, buf, F, nullptr) == MX_OK);
        CHECK(mx::norm.ld_x == ld * (src ? 2 : 4) && mx::norm.cols == cols && mx::norm.fmt == fmt);
        const int64_t need = mx_rmsnorm_backward_workspace(3, cols, src);
        CHECK(need == 3 * cols * 4);
        CHECK(mx_rmsnorm_backward(P, ld, P, ld, P, F, nullptr, 0, 3, cols, src, P, ld, F, P, need, nullptr) == MX_OK);
        CHECK(mx::grad.dh == nullptr && mx::grad.rows == 3);
      }
  CHECK(mx_rmsnorm_backward(nullptr, 0, nullptr, 0, nullptr, nullptr, nullptr, 0, 0, 64, 0, nullptr, 0, F, nullptr, 0,
                            nullptr) == MX_OK);
  CHECK(mx::grad.rows == 0);
  for (int64_t K : {0, 1, 33, 4096}) {
    CHECK(mx_gemv(P, K, P, buf, MX_E2M1, 3, 7, K, F, 7, nullptr) == MX_OK && !mx::gemv.bf16 && mx::gemv.K == K);
    CHECK(mx_gemv_bf16(buf + 2, K, P, buf, MX_E2M1, 3, 7, K, (uint16_t*)(buf + 2), 9, nullptr) == MX_OK && mx::gemv.bf16);
  }
  CHECK(mx_gemv(P, big, P, buf, MX_E2M1, 3, 7, 64, F, big, nullptr) == MX_OK);
  CHECK(mx_gemv(P, big, P, buf, MX_E2M1, 3, 7, big, F, 7, nullptr) == MX_ERR_UNSUPPORTED);
  mx_cache c;
  std::memset(&c, 0, sizeof c);
  c.k_q = c.v_q = P;
  c.k_s = c.v_s = buf;
  c.pages = 5;
  c.heads = 2;
  c.page = 48;
  for (int dim : {64, 128, 256}) {
    c.dim = dim;
    for (int fmt = 0; fmt < 2; fmt++) {
      c.fmt = fmt;
      CHECK(mx_cache_write(&c, P, 2 * dim, dim, P, 0, 0, MX_SRC_F32, 9, (const int64_t*)P, nullptr) == MX_OK);
      CHECK(mx::cwrite.ld_k == 8 * dim && mx::cwrite.ld_v == 0 && mx::cwrite.c.page == 48);
      CHECK(mx_attention(&c, P, 6 * dim, (const int32_t*)P, 3, (const int32_t*)P, 2, 3, 6, 1.0f, 144, (uint16_t*)P, 6 * dim,
                         nullptr, nullptr, 0, nullptr) == MX_ERR_HIP);  // the stub's refusal
      CHECK(mx::att.group == 3 && mx::att.max_len == 144 && mx::att.lse == nullptr);
    }
  }
  c.pages = 0;  // nothing to read: no token is looked for
  c.k_q = nullptr;
  CHECK(mx_attention(&c, P, 6 * 256, (const int32_t*)P, 3, (const int32_t*)P, 2, 3, 6, 1.0f, 144, (uint16_t*)P, 6 * 256,
                     nullptr, nullptr, 0, nullptr) == MX_ERR_HIP);
  CHECK(mx::att.max_len == 0);
  CHECK(mx_attention_workspace(2, 1, 6, 2, 64, 2000) == 4096);
  CHECK(mx_attention_workspace(big, 1, 6, 2, 64, 2000) == -1 && mx_attention_workspace(2, big, 6, 2, 64, 9) == -1);
  CHECK(mx_attention_workspace(2, 1, big, 1, 64, 9) == -1 && mx_attention_workspace(2, 1, 6, 2, 64, big) == -1);
  if (fails) return 1;
  std::printf("layer entry points: %d launcher calls, all checks passed\n", mx::calls);
  return 0;
}
