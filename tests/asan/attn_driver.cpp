// Host-side driver for the AddressSanitizer build of the attention and cache entry points (tests/test_asan_attn.py):
// argument validation of valid and invalid calls in dry-run mode.  The launchers are stubs that abort, and the shared
// helpers of the library are small stand-ins.  Exit status 0 and no sanitizer report is a pass.
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "mxfp8.h"

struct ihipStream_t;
typedef ihipStream_t* hipStream_t;

#define STUB                                                            \
  {                                                                     \
    std::fprintf(stderr, "a launcher was reached in dry-run mode\n");   \
    std::abort();                                                       \
  }

static char g_err[512];

namespace mx {
enum Counter : int;
mx_status fail(mx_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return st;
}
void clear_error() { g_err[0] = 0; }
bool dry_run() { return true; }
mx_status require_gfx950() STUB
struct KvCache;
mx_status launch_kv_write(const void*, int64_t, const void*, int64_t, int64_t, int32_t, int32_t, const int64_t*, bool,
                          void*, uint8_t*, void*, uint8_t*, int64_t, uint32_t, hipStream_t) STUB
mx_status launch_kv_read(const KvCache&, bool, int32_t, int64_t, const int32_t*, int64_t, void*, void*, hipStream_t) STUB
size_t decode_workspace_bytes(int64_t B, int32_t H, int32_t, int32_t D, int64_t) { return static_cast<size_t>(B) * H * D; }
mx_status launch_attn_decode(const void*, int64_t, int64_t, int32_t, int32_t, bool, const KvCache&, const int32_t*, float,
                             void*, void*, hipStream_t) STUB
size_t prefill_workspace_bytes(int64_t, int64_t Tq, int64_t, int32_t H, int32_t, int32_t D) {
  return static_cast<size_t>(Tq) * H * D;
}
mx_status launch_attn_prefill(const void*, int64_t, const void*, int64_t, const void*, int64_t, const int32_t*,
                              const int32_t*, int64_t, int64_t, int64_t, int32_t, int32_t, int32_t, float, void*, void*,
                              hipStream_t) STUB
}  // namespace mx
// mx::count(Counter), whose enumeration the library keeps to itself
extern "C" void _ZN2mx5countENS_7CounterE(int) STUB

static int failures = 0;
#define EXPECT(cond)                                                                          \
  do {                                                                                        \
    if (!(cond)) {                                                                            \
      std::fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__, __LINE__, #cond);     \
      ++failures;                                                                             \
    }                                                                                         \
  } while (0)

int main() {
  uint8_t* const p = reinterpret_cast<uint8_t*>(uintptr_t(1) << 20);
  const int64_t* const slots = reinterpret_cast<const int64_t*>(p);
  const int32_t* const ints = reinterpret_cast<const int32_t*>(p);
  const int64_t big = INT64_MAX;
  const size_t all = SIZE_MAX;

  auto write = [&](int64_t T, int32_t Hkv, int32_t D, int64_t stride, int64_t pages, int32_t page) {
    return mx_kv_cache_write(p, stride, p, stride, T, Hkv, D, slots, MX_CACHE_MXFP8, p, p, p, p, pages, page, nullptr);
  };
  auto read = [&](int64_t B, int64_t max_pages, int64_t rows, int32_t Hkv, int32_t D) {
    return mx_kv_cache_read(MX_CACHE_BF16, p, nullptr, p, nullptr, 10, 64, Hkv, D, ints, B, max_pages, ints, rows, p, p, nullptr);
  };
  auto decode = [&](int64_t B, int32_t H, int32_t Hkv, int32_t D, int64_t max_pages, int64_t stride, float scale) {
    return mx_attn_decode(p, stride, B, H, Hkv, D, MX_CACHE_MXFP8, p, p, nullptr, nullptr, 10, 64, ints, max_pages, ints, scale, p, p,
                          all, nullptr);
  };
  auto prefill = [&](int64_t B, int64_t Tq, int64_t Tk, int32_t H, int32_t Hkv, int64_t stride) {
    return mx_attn_prefill(p, stride, p, 1024, p, 1024, ints, ints, B, Tq, Tk, H, Hkv, 128, 0.1f, p, p, all, nullptr);
  };

  EXPECT(write(100, 4, 128, 512, 10, 64) == MX_OK);
  EXPECT(read(3, 7, 100, 4, 128) == MX_OK);
  EXPECT(decode(5, 8, 4, 128, 7, 1024, 0.1f) == MX_OK);
  EXPECT(prefill(3, 1000, 2000, 8, 4, 1024) == MX_OK);
  EXPECT(write(0, 4, 128, 512, 10, 64) == MX_OK && read(0, 7, 100, 4, 128) == MX_OK && decode(0, 8, 4, 128, 7, 1024, 0.1f) == MX_OK &&
         prefill(0, 0, 0, 8, 4, 1024) == MX_OK);

  // the ends of every argument's range
  for (int64_t x : {-big - 1, int64_t(-1), big, big / 2, int64_t(1) << 33}) {
    EXPECT(write(x, 4, 128, 512, 10, 64) == MX_ERR_INVALID_ARG);
    EXPECT(write(100, 4, 128, x, 10, 64) == MX_ERR_INVALID_ARG);
    EXPECT(write(100, 4, 128, 512, x, 64) == MX_ERR_INVALID_ARG);
    EXPECT(read(x, 7, 100, 4, 128) == MX_ERR_INVALID_ARG);
    EXPECT(read(3, x, 100, 4, 128) == MX_ERR_INVALID_ARG);
    EXPECT(read(3, 7, x, 4, 128) == MX_ERR_INVALID_ARG);
    EXPECT(decode(x, 8, 4, 128, 7, 1024, 0.1f) == MX_ERR_INVALID_ARG);
    EXPECT(decode(5, 8, 4, 128, x, 1024, 0.1f) == MX_ERR_INVALID_ARG);
    EXPECT(decode(5, 8, 4, 128, 7, x, 0.1f) == MX_ERR_INVALID_ARG);
    EXPECT(prefill(x, 1000, 2000, 8, 4, 1024) == MX_ERR_INVALID_ARG);
    EXPECT(prefill(3, x, 2000, 8, 4, 1024) == MX_ERR_INVALID_ARG);
    EXPECT(prefill(3, 1000, x, 8, 4, 1024) == MX_ERR_INVALID_ARG);
    EXPECT(prefill(3, 1000, 2000, 8, 4, x) == MX_ERR_INVALID_ARG);
    EXPECT(mx_attn_decode_workspace_bytes(x, 8, 4, 128, 7, 64) == 0);
    EXPECT(mx_attn_decode_workspace_bytes(5, 8, 4, 128, x, 64) == 0);
    EXPECT(mx_attn_prefill_workspace_bytes(x, 10, 10, 8, 4, 128) == 0);
    EXPECT(mx_attn_prefill_workspace_bytes(1, x, 10, 8, 4, 128) == 0);
    EXPECT(mx_attn_prefill_workspace_bytes(1, 10, x, 8, 4, 128) == 0);
  }
  for (int32_t x : {INT32_MIN, -1, 0, INT32_MAX, 1 << 30}) {
    EXPECT(write(100, x, 128, 512, 10, 64) == MX_ERR_INVALID_ARG);
    EXPECT(write(100, 4, x, 512, 10, 64) == MX_ERR_INVALID_ARG);
    EXPECT(write(100, 4, 128, 512, 10, x) == MX_ERR_INVALID_ARG);
    EXPECT(read(3, 7, 100, x, 128) == MX_ERR_INVALID_ARG);
    EXPECT(read(3, 7, 100, 4, x) == MX_ERR_INVALID_ARG);
    EXPECT(decode(5, x, 4, 128, 7, 1024, 0.1f) == MX_ERR_INVALID_ARG);
    EXPECT(decode(5, 8, x, 128, 7, 1024, 0.1f) == MX_ERR_INVALID_ARG);
    EXPECT(decode(5, 8, 4, x, 7, 1024, 0.1f) == MX_ERR_INVALID_ARG);
    EXPECT(prefill(3, 1000, 2000, x, 4, 1024) == MX_ERR_INVALID_ARG);
    EXPECT(prefill(3, 1000, 2000, 8, x, 1024) == MX_ERR_INVALID_ARG);
    EXPECT(mx_attn_decode_workspace_bytes(5, 8, x, 128, 7, 64) == 0);
    EXPECT(mx_attn_decode_workspace_bytes(5, x, 4, 128, 7, 64) == 0);
    EXPECT(mx_attn_prefill_workspace_bytes(1, 10, 10, 8, x, 128) == 0);
  }
  if (!failures) std::printf("all checks passed\n");
  return failures ? 1 : 0;
}
