// C ABI of the mixture-of-experts operators and the block-128 linear: argument validation and dispatch, by the rules of
// api.hip (checks before the GPU is touched, nothing throws).
#include <algorithm>

#include "api_checks.hpp"

namespace mx {

size_t route_workspace_bytes(int64_t T, int32_t E);
mx_status launch_moe_route(const void* logits, int32_t f32, const float* bias, int64_t T, int32_t E, int32_t k,
                           int32_t score, int32_t renormalize, float scale, int32_t* ids, float* weights,
                           int32_t* offsets, int32_t* row_slot, int32_t* slot_row, void* workspace,
                           hipStream_t stream);
mx_status launch_moe_combine(const void* y, int64_t rows, int64_t N, const int32_t* slot_row, const float* weights,
                             int64_t T, int32_t k, const void* shared, void* out, hipStream_t stream);
size_t grouped_workspace_bytes(int64_t rows, int64_t S, int64_t E, int64_t N, int64_t K);
mx_status launch_grouped(const void* x, int64_t rows, const uint8_t* w, const void* ws, bool f32, bool act,
                         const int32_t* offsets, const int32_t* row_slot, int32_t k, int64_t S, int64_t E, int64_t N,
                         int64_t K, void* out, void* workspace, hipStream_t stream, const char* what);

}  // namespace mx

using namespace mx;

extern "C" {

size_t mx_moe_route_workspace_bytes(int64_t T, int32_t E) {
  if (T <= 0 || E <= 0) return 0;
  return route_workspace_bytes(T, E);
}

mx_status mx_moe_route(const void* logits, int32_t logits_f32, const float* bias, int64_t T, int32_t E, int32_t k,
                       int32_t score, int32_t renormalize, float scale, int32_t* ids, float* weights,
                       int32_t* offsets, int32_t* row_slot, int32_t* slot_row, void* workspace,
                       size_t workspace_bytes, void* stream) {
  const char* fn = "mx_moe_route";
  MX_CHECK(logits_f32 == 0 || logits_f32 == 1, "%s: logits_f32 = %d (0 or 1)", fn, logits_f32);
  MX_CHECK(E >= 1 && E <= MX_ROUTE_MAX_EXPERTS, "%s: E = %d (1 to %d)", fn, E, MX_ROUTE_MAX_EXPERTS);
  MX_CHECK(k >= 1 && k <= std::min(E, MX_ROUTE_MAX_K), "%s: k = %d (1 to min(E = %d, %d))", fn, k, E,
           MX_ROUTE_MAX_K);
  // a workgroup of 512 threads takes 64 tokens, and a launch is below 2^32 threads
  MX_CHECK(T >= 0 && T < (int64_t(1) << 29) - 64 && T * k < (int64_t(1) << 31), "%s: T = %lld out of range", fn,
           (long long)T);
  MX_CHECK(score == MX_ROUTE_SOFTMAX || score == MX_ROUTE_SIGMOID, "%s: unknown score %d", fn, score);
  MX_CHECK(renormalize == 0 || renormalize == 1, "%s: renormalize = %d (0 or 1)", fn, renormalize);
  MX_CHECK(offsets && aligned(offsets, 4), "%s: offsets must be a 4-byte aligned pointer", fn);
  if (T > 0) {
    MX_CHECK(logits && ids && weights && row_slot && slot_row, "%s: null tensor pointer", fn);
    MX_CHECK(aligned(logits, logits_f32 ? 4 : 2) && aligned(bias, 4) && aligned(ids, 4) && aligned(weights, 4) &&
                 aligned(row_slot, 4) && aligned(slot_row, 4),
             "%s: logits must be aligned to their element, the other tensors to 4 bytes", fn);
    const size_t need = mx_moe_route_workspace_bytes(T, E);
    MX_CHECK(workspace_bytes >= need && (need == 0 || (workspace && aligned(workspace, 8))),
             "%s: workspace of %zu bytes (8-byte aligned) needed, got %zu", fn, need, workspace_bytes);
  }
  // The kernels read ids and the workspace back as indices, so nothing may have been written over them.  (Not in a dry
  // run, whose pointers are stand-ins.)
  if (!dry_run()) {
    const size_t n = static_cast<size_t>(T), slots = n * k * 4;
    const struct { const char* name; const void* at; size_t bytes; } part[] = {
        {"ids", ids, slots}, {"weights", weights, slots}, {"row_slot", row_slot, slots}, {"slot_row", slot_row, slots},
        {"offsets", offsets, (static_cast<size_t>(E) + 1) * 4},
        {"workspace", workspace, mx_moe_route_workspace_bytes(T, E)},
        {"logits", logits, n * E * (logits_f32 ? 4 : 2)}, {"bias", bias, static_cast<size_t>(E) * 4}};
    for (int i = 0; i < 6; ++i)
      for (int j = i + 1; j < 8; ++j)
        MX_CHECK(apart(part[i].at, part[i].bytes, part[j].at, part[j].bytes), "%s: %s overlaps %s", fn, part[i].name,
                 part[j].name);
  }
  MX_PREAMBLE();
  count(C_MOE_ROUTE);
  const mx_status st = launch_moe_route(logits, logits_f32, bias, T, E, k, score, renormalize, scale, ids, weights,
                                        offsets, row_slot, slot_row, workspace, static_cast<hipStream_t>(stream));
  if (st == MX_OK) clear_error();
  return st;
}

mx_status mx_moe_combine(const void* y, int64_t rows, int64_t N, const int32_t* slot_row, const float* weights,
                         int64_t T, int32_t k, const void* shared, void* out, void* stream) {
  const char* fn = "mx_moe_combine";
  MX_CHECK(T >= 0 && rows >= 0 && rows < (int64_t(1) << 31), "%s: T = %lld, rows = %lld out of range", fn,
           (long long)T, (long long)rows);
  MX_CHECK(N >= 8 && N % 8 == 0 && N < (int64_t(1) << 31), "%s: N = %lld is not a positive multiple of 8", fn,
           (long long)N);
  MX_CHECK(k >= 1 && k <= 1024, "%s: k = %d (1 to 1024)", fn, k);
  // a thread takes 8 elements, and a launch is below 2^32 threads
  MX_CHECK(T < (int64_t(1) << 31) && T * N <= (int64_t(1) << 35) - 2048, "%s: T = %lld x N = %lld too large", fn,
           (long long)T, (long long)N);
  if (T == 0) { clear_error(); return MX_OK; }
  MX_CHECK((y || rows == 0) && slot_row && weights && out, "%s: null tensor pointer", fn);
  MX_CHECK(aligned(y, 16) && aligned(shared, 16) && aligned(out, 16) && aligned(slot_row, 4) && aligned(weights, 4),
           "%s: y, shared and out must be 16-byte, slot_row and weights 4-byte aligned", fn);
  const size_t out_bytes = static_cast<size_t>(T) * N * 2, slot_bytes = static_cast<size_t>(T) * k * 4;
  MX_CHECK(apart(out, out_bytes, y, static_cast<size_t>(rows) * N * 2), "%s: out overlaps y", fn);
  MX_CHECK(shared == out || apart(out, out_bytes, shared, out_bytes), "%s: out overlaps shared without being it", fn);
  MX_CHECK(apart(out, out_bytes, slot_row, slot_bytes) && apart(out, out_bytes, weights, slot_bytes),
           "%s: out overlaps slot_row or weights", fn);
  MX_PREAMBLE();
  count(C_MOE_COMBINE);
  const mx_status st =
      launch_moe_combine(y, rows, N, slot_row, weights, T, k, shared, out, static_cast<hipStream_t>(stream));
  if (st == MX_OK) clear_error();
  return st;
}

}  // extern "C"

namespace {

// Argument checks shared by mx_grouped_linear and mx_linear_block128: `rows` rows of x, S of out.
mx_status grouped_check(const char* fn, const void* x, int64_t rows, int64_t x_width, int64_t K, const void* w,
                        const void* w_scale, bool f32, const int32_t* offsets, const int32_t* row_slot, int64_t E,
                        int64_t N, int64_t S, const void* out, const void* workspace, size_t workspace_bytes,
                        size_t need) {
  MX_CHECK(x && w && w_scale && out, "%s: null tensor pointer", fn);
  MX_CHECK(aligned(x, 16) && aligned(w, 16) && aligned(out, 16), "%s: x, w and out must be 16-byte aligned", fn);
  MX_CHECK(!f32 || aligned(w_scale, 4), "%s: FP32 w_scale must be 4-byte aligned", fn);
  MX_CHECK(workspace && aligned(workspace, 16) && workspace_bytes >= need,
           "%s: workspace of %zu bytes (16-byte aligned) needed, got %zu", fn, need, workspace_bytes);
  const struct { const char* name; const void* at; int64_t bytes; } in[] = {
      {"x", x, rows * x_width * 2}, {"w", w, E * N * K},
      {"w_scale", w_scale, f32 ? E * ((N + 127) / 128) * ((K + 127) / 128) * 4 : E * N * (K / MX_LINEAR_BLOCK)},
      {"offsets", offsets, (E + 1) * 4}, {"row_slot", row_slot, S * 4}};
  MX_CHECK(apart(out, S * N * 2, workspace, need), "%s: out overlaps the workspace", fn);
  for (const auto& t : in) {
    MX_CHECK(apart(out, S * N * 2, t.at, t.bytes), "%s: out overlaps %s", fn, t.name);
    // The list of row tiles and the codes are written while the offsets and x are read.  (Not in a dry run, whose
    // pointers are stand-ins.)
    MX_CHECK(dry_run() || apart(workspace, need, t.at, t.bytes), "%s: the workspace overlaps %s", fn, t.name);
  }
  return MX_OK;
}

// Sizes both take.
mx_status grouped_sizes(const char* fn, int64_t rows, int64_t K, bool f32, int64_t E, int64_t N, int64_t S) {
  const int64_t step = f32 ? 16 : MX_LINEAR_BLOCK;
  MX_CHECK(rows >= 0 && S >= 0 && S < (int64_t(1) << 31), "%s: rows = %lld, S = %lld out of range", fn,
           (long long)rows, (long long)S);
  MX_CHECK(K >= 16 && K % step == 0 && K < (int64_t(1) << 22), "%s: K = %lld is not a multiple of %lld below 2^22", fn,
           (long long)K, (long long)step);
  MX_CHECK(N >= 16 && N % 16 == 0 && N < (int64_t(1) << 31), "%s: N = %lld is not a positive multiple of 16", fn,
           (long long)N);
  MX_CHECK(E >= 1 && E < (int64_t(1) << 20), "%s: E = %lld out of range", fn, (long long)E);
  const int64_t Kp = (K + 127) / 128 * 128;
  MX_CHECK(rows < (int64_t(1) << 31) && rows * Kp < (int64_t(1) << 32) - 256,
           "%s: rows * K = %lld x %lld too large for 32-bit row offsets", fn, (long long)rows, (long long)K);
  // A launch of the tiles (256 threads for 128 x 128, 512 for 256 x 256) is below 2^32 threads, and the 32 x 16 units that
  // the smallest tiles are cut into are numbered with 31 bits.
  MX_CHECK((S / 128 + std::min(S, E)) * ((N + 127) / 128) < (int64_t(1) << 23) - 512, "%s: S = %lld x N = %lld too large", fn,
           (long long)S, (long long)N);
  return MX_OK;
}

}  // namespace

extern "C" {

size_t mx_grouped_linear_workspace_bytes(int64_t rows, int64_t S, int64_t E, int64_t N, int64_t K) {
  if (rows <= 0 || S <= 0 || E <= 0 || N <= 0 || K <= 0) return 0;
  return grouped_workspace_bytes(rows, S, E, N, K);
}

mx_status mx_grouped_linear(const void* x, int64_t rows, int64_t K, const uint8_t* w, const void* w_scale,
                            int32_t scale_kind, int64_t E, int64_t N, const int32_t* offsets,
                            const int32_t* row_slot, int32_t k, int64_t S, int32_t act, void* out, void* workspace,
                            size_t workspace_bytes, void* stream) {
  const char* fn = "mx_grouped_linear";
  MX_CHECK(scale_kind == MX_SCALE_E8M0 || scale_kind == MX_SCALE_F32, "%s: unknown scale kind %d", fn, scale_kind);
  MX_CHECK(act == MX_ACT_NONE || act == MX_ACT_SWIGLU, "%s: unknown act %d", fn, act);
  MX_CHECK(k >= 1, "%s: k = %d < 1", fn, k);
  const bool f32 = scale_kind == MX_SCALE_F32;
  mx_status st = grouped_sizes(fn, rows, K, f32, E, N, S);
  if (st != MX_OK) return st;
  MX_CHECK(row_slot || S == rows, "%s: without row_slot the rows of x (%lld) are the rows of out (%lld)", fn,
           (long long)rows, (long long)S);
  if (S == 0) { clear_error(); return MX_OK; }
  MX_CHECK(rows >= 1, "%s: x has no rows", fn);
  MX_CHECK(offsets && aligned(offsets, 4) && aligned(row_slot, 4),
           "%s: offsets and row_slot must be 4-byte aligned, offsets not null", fn);
  st = grouped_check(fn, x, rows, act == MX_ACT_SWIGLU ? 2 * K : K, K, w, w_scale, f32, offsets, row_slot, E, N, S,
                     out, workspace, workspace_bytes, mx_grouped_linear_workspace_bytes(rows, S, E, N, K));
  if (st != MX_OK) return st;
  MX_PREAMBLE();
  count(C_GROUPED_LINEAR);
  st = launch_grouped(x, rows, w, w_scale, f32, act == MX_ACT_SWIGLU, offsets, row_slot, k, S, E, N, K, out,
                      workspace, static_cast<hipStream_t>(stream), fn);
  if (st == MX_OK) clear_error();
  return st;
}

size_t mx_linear_block128_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return mx_grouped_linear_workspace_bytes(M, M, 1, N, K);
}

mx_status mx_linear_block128(const void* x, int64_t M, int64_t K, const uint8_t* w, const float* w_scale, int64_t N,
                             void* out, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "mx_linear_block128";
  mx_status st = grouped_sizes(fn, M, K, true, 1, N, M);
  if (st != MX_OK) return st;
  if (M == 0) { clear_error(); return MX_OK; }
  st = grouped_check(fn, x, M, K, K, w, w_scale, true, nullptr, nullptr, 1, N, M, out, workspace, workspace_bytes,
                     mx_linear_block128_workspace_bytes(M, N, K));
  if (st != MX_OK) return st;
  MX_PREAMBLE();
  count(C_LINEAR_BLOCK128);
  st = launch_grouped(x, M, w, w_scale, true, false, nullptr, nullptr, 1, M, 1, N, K, out, workspace,
                      static_cast<hipStream_t>(stream), fn);
  if (st == MX_OK) clear_error();
  return st;
}

}  // extern "C"
