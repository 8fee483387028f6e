// Host-side driver for the AddressSanitizer build of the mixture-of-experts entry points (tests/test_asan_moe.py):
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
size_t route_workspace_bytes(int64_t T, int32_t E) { return T > 64 ? static_cast<size_t>(T / 64 + 1) * E * 4 : 0; }
size_t grouped_workspace_bytes(int64_t rows, int64_t, int64_t, int64_t, int64_t K) { return rows * (K + 128); }
mx_status launch_moe_route(const void*, int32_t, const float*, int64_t, int32_t, int32_t, int32_t, int32_t, float,
                           int32_t*, float*, int32_t*, int32_t*, int32_t*, void*, hipStream_t) STUB
mx_status launch_moe_combine(const void*, int64_t, int64_t, const int32_t*, const float*, int64_t, int32_t,
                             const void*, void*, hipStream_t) STUB
mx_status launch_grouped(const void*, int64_t, const uint8_t*, const void*, bool, bool, const int32_t*,
                         const int32_t*, int32_t, int64_t, int64_t, int64_t, int64_t, void*, void*, hipStream_t,
                         const char*) STUB
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
  uint8_t* const q = reinterpret_cast<uint8_t*>(uintptr_t(1) << 44);
  uint8_t* const r = reinterpret_cast<uint8_t*>(uintptr_t(1) << 45);
  int32_t* const i = reinterpret_cast<int32_t*>(p);
  float* const f = reinterpret_cast<float*>(p);
  const size_t big = size_t(1) << 40;
  for (int64_t T : {int64_t(0), int64_t(1), int64_t(1) << 20, int64_t(1) << 40, int64_t(-5)})
    for (int32_t E : {0, 1, 1024, 1025, -1})
      for (int32_t k : {0, 1, 32, 33, INT32_MAX}) {
        const bool ok = T >= 0 && T < (int64_t(1) << 31) && E >= 1 && E <= 1024 && k >= 1 && k <= 32 && k <= E &&
                        T * k < (int64_t(1) << 31);
        EXPECT((mx_moe_route(p, 1, f, T, E, k, 0, 1, 1.f, i, f, i, i, i, p, big, nullptr) == MX_OK) == ok);
      }
  for (int64_t rows : {int64_t(0), int64_t(1), int64_t(1) << 20, int64_t(1) << 40, int64_t(-1)})
    for (int64_t K : {int64_t(0), int64_t(16), int64_t(32), int64_t(4096), INT64_MAX / 2})
      for (int64_t N : {int64_t(16), int64_t(24), int64_t(1) << 31, int64_t(-16)}) {
        const bool ok = rows >= 0 && rows < (int64_t(1) << 31) && K >= 32 && K <= 4096 && N == 16 &&
                        rows * ((K + 127) / 128 * 128) < (int64_t(1) << 32) - 256;
        EXPECT((mx_grouped_linear(p, rows, K, q, p, 0, 4, N, i, nullptr, 1, rows, 0, r, p, big, nullptr) == MX_OK) ==
               ok);
        const bool okd = rows >= 0 && rows < (int64_t(1) << 31) && K >= 16 && K <= 4096 && N == 16 &&
                         rows * ((K + 127) / 128 * 128) < (int64_t(1) << 32) - 256;
        EXPECT((mx_linear_block128(p, rows, K, q, f, N, r, p, big, nullptr) == MX_OK) == okd);
        EXPECT(mx_grouped_linear_workspace_bytes(-1, 4, 4, N, K) == 0);
      }
  for (int64_t T : {int64_t(0), int64_t(7), int64_t(1) << 31, int64_t(-1)})
    EXPECT((mx_moe_combine(p, 100, 512, i, f, T, 8, q, r, nullptr) == MX_OK) == (T >= 0 && T < 8));
  if (failures) return 1;
  std::printf("all checks passed\n");
  return 0;
}
