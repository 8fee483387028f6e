// Host-side driver for the sanitizer build of the attention calls' workspace sizes (tests/test_asan_attn.py): the library's
// own arithmetic, over the ends of every argument's range and their products, in dry-run mode.  The launchers are linked in
// but never reached; the HIP runtime is stubs.  Exit status 0 and no sanitizer report is a pass.
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "mxfp8.h"

#define STUB                                                          \
  {                                                                   \
    std::fprintf(stderr, "the GPU was reached in dry-run mode\n");    \
    std::abort();                                                     \
  }

namespace mx {
enum Counter : int;
mx_status fail(mx_status st, const char*, ...) { return st; }
void clear_error() {}
bool dry_run() { return true; }
mx_status require_gfx950() STUB
mx_status launch_status(const char*) STUB
}  // namespace mx
extern "C" {
void _ZN2mx5countENS_7CounterE(int) STUB     // mx::count(Counter), whose enumeration the library keeps to itself
// what a HIP object registers when it is loaded, and launches with
void** __hipRegisterFatBinary(const void*) { return nullptr; }
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, void*, void*, int*) {}
void __hipUnregisterFatBinary(void**) {}
int __hipPushCallConfiguration() STUB
int __hipPopCallConfiguration() STUB
int hipLaunchKernel() STUB
}

static int failures = 0;
#define EXPECT(cond, ...)                       \
  do {                                          \
    if (!(cond) && ++failures < 20) {           \
      std::printf("%s: ", #cond);               \
      std::printf(__VA_ARGS__);                 \
      std::printf("\n");                        \
    }                                           \
  } while (0)

int main() {
  uint8_t* const p = reinterpret_cast<uint8_t*>(uintptr_t(1) << 20);
  const int32_t* const ints = reinterpret_cast<const int32_t*>(p);
  const std::vector<int64_t> counts = {INT64_MIN, -1, 0, 1, 63, 64, 129, 4099, 65536, 1 << 20, (1 << 23) - 1, 1 << 23, (1 << 24) - 16384,
                                       (1 << 24) - 1, 1 << 24, 1 << 27, 1 << 30, (int64_t(1) << 31) - 65, (int64_t(1) << 31) - 1,
                                       int64_t(1) << 31, int64_t(1) << 33, INT64_MAX / 2, INT64_MAX};
  const std::vector<int32_t> heads = {INT32_MIN, -1, 0, 1, 2, 3, 48, 128, 4095, 65535, 65536, 65537, INT32_MAX};
  const std::vector<int32_t> widths = {INT32_MIN, -1, 0, 32, 64, 96, 128, 256, 512, 1024, INT32_MAX};
  const std::vector<int32_t> pages = {INT32_MIN, -1, 0, 8, 16, 48, 64, 4096, 8192, INT32_MAX};
  long accepted = 0, calls = 0;

  // a call with all the memory there is passes where, and only where, its workspace has a size, and not with a byte less
  for (int64_t B : counts)
    for (int32_t H : heads)
      for (int32_t Hkv : heads)
        for (int32_t D : widths) {
          for (int64_t n : counts)
            for (int32_t page : pages) {
              const size_t need = mx_attn_decode_workspace_bytes(B, H, Hkv, D, n, page);
              auto call = [&](size_t bytes) {
                return mx_attn_decode(p, int64_t(H) * D, B, H, Hkv, D, MX_CACHE_BF16, p, nullptr, p, nullptr, 1, page, ints, n, ints,
                                      0.1f, p, p, bytes, nullptr);
              };
              ++calls;
              if (B == 0) {
                EXPECT(need == 0, "H %d Hkv %d D %d", H, Hkv, D);
                continue;
              }
              EXPECT((call(SIZE_MAX) == MX_OK) == (need != 0), "decode B %lld H %d Hkv %d D %d max_pages %lld page %d", (long long)B, H,
                     Hkv, D, (long long)n, page);
              if (need != 0) {
                ++accepted;
                EXPECT(call(need) == MX_OK && call(need - 1) == MX_ERR_INVALID_ARG, "decode B %lld H %d: %zu bytes", (long long)B, H, need);
                EXPECT(need < (size_t(1) << 36), "decode B %lld H %d Hkv %d D %d: %zu bytes", (long long)B, H, Hkv, D, need);
              }
            }
          for (int64_t Tq : counts)
            for (int64_t Tk : counts) {
              const size_t need = mx_attn_prefill_workspace_bytes(B, Tq, Tk, H, Hkv, D);
              auto call = [&](size_t bytes) {
                return mx_attn_prefill(p, int64_t(H) * D, p, int64_t(Hkv) * D, p, int64_t(Hkv) * D, ints, ints, B, Tq, Tk, H, Hkv, D,
                                       0.1f, p, p, bytes, nullptr);
              };
              ++calls;
              if (need == 0) {
                if (B != 0 && Tq != 0) EXPECT(call(0) == call(SIZE_MAX), "prefill B %lld Tq %lld", (long long)B, (long long)Tq);
                continue;
              }
              ++accepted;
              EXPECT(call(need) == MX_OK && call(need - 1) == MX_ERR_INVALID_ARG, "prefill B %lld Tq %lld Tk %lld H %d Hkv %d D %d: %zu bytes",
                     (long long)B, (long long)Tq, (long long)Tk, H, Hkv, D, need);
              EXPECT(need < (size_t(1) << 36), "prefill B %lld Tq %lld Tk %lld H %d: %zu bytes", (long long)B, (long long)Tq, (long long)Tk, H, need);
            }
        }
  if (!failures) std::printf("all checks passed: %ld sizes, %ld of them with a workspace\n", calls, accepted);
  return failures ? 1 : 0;
}
