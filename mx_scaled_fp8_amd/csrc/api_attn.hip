// C ABI of the key-value cache and the attention over it: argument validation and dispatch, by the rules of api.hip
// (checks before the GPU is touched, nothing throws).
#include <cmath>

#include "api_checks.hpp"
#include "kv_cache.hpp"

namespace mx {

mx_status launch_kv_write(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t T, int32_t Hkv,
                          int32_t D, const int64_t* slots, bool fp8, void* k_cache, uint8_t* k_scale, void* v_cache,
                          uint8_t* v_scale, int64_t pages, uint32_t page_shift, hipStream_t stream);
mx_status launch_kv_read(const KvCache& c, bool fp8, int32_t D, int64_t B, const int32_t* offsets, int64_t rows,
                         void* k, void* v, hipStream_t stream);
size_t decode_workspace_bytes(int64_t B, int32_t H, int32_t Hkv, int32_t D, int64_t max_tokens);
mx_status launch_attn_decode(const void* q, int64_t q_stride, int64_t B, int32_t H, int32_t D, bool fp8,
                             const KvCache& c, const int32_t* lens, float scale, void* out, void* workspace,
                             hipStream_t stream);
size_t prefill_workspace_bytes(int64_t B, int64_t Tq, int64_t Tk, int32_t H, int32_t Hkv, int32_t D);
mx_status launch_attn_prefill(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, const int32_t* q_offsets, const int32_t* k_offsets, int64_t B,
                              int64_t Tq, int64_t Tk, int32_t H, int32_t Hkv, int32_t D, float scale, void* out,
                              void* workspace, hipStream_t stream);

}  // namespace mx

using namespace mx;

namespace {

constexpr int64_t k31 = int64_t(1) << 31;

struct Span { const char* name; const void* at; size_t bytes; };

// The first n spans are written: they overlap neither each other nor any other.  (Not in a dry run, whose pointers are
// stand-ins.)
mx_status check_apart(const char* fn, const Span* part, int written, int n) {
  if (dry_run()) return MX_OK;
  for (int i = 0; i < written; ++i)
    for (int j = i + 1; j < n; ++j)
      MX_CHECK(apart(part[i].at, part[i].bytes, part[j].at, part[j].bytes), "%s: %s overlaps %s", fn, part[i].name,
               part[j].name);
  return MX_OK;
}

// Bytes from the first to the last element of n strided rows.
size_t extent(int64_t n, int64_t stride, int64_t width) {
  return n > 0 ? (static_cast<size_t>(n - 1) * stride + width) * 2 : 0;
}

bool head_dim(int32_t D) { return D == 64 || D == 128 || D == 256 || D == 512; }
bool heads_fit(int32_t H, int32_t Hkv) { return Hkv >= 1 && H >= 1 && H <= 65536 && H % Hkv == 0; }
bool page_fits(int32_t page_size) {
  return page_size >= 16 && page_size <= MX_CACHE_MAX_PAGE && (page_size & (page_size - 1)) == 0;
}
bool row_fits(int32_t Hkv, int32_t D) {
  return Hkv >= 1 && D >= 32 && D <= 1024 && D % MX_CACHE_BLOCK == 0 && int64_t(Hkv) * D <= (int64_t(1) << 20);
}

// The sizes of a call, each and their products, of heads (and pages) that fit: what the call and the query of its workspace
// agree on, and what keeps the launchers' arithmetic in range.
bool decode_fits(int64_t B, int32_t H, int32_t Hkv, int64_t max_pages, int32_t page_size) {
  if (B < 0 || B >= (int64_t(1) << 24) || max_pages < 1 || max_pages >= k31 || max_pages * page_size >= k31) return false;
  const int64_t streams = B * Hkv * ((H / Hkv + 15) / 16);
  return streams < (int64_t(1) << 24) && streams * ((max_pages * page_size + 31) / 32) < k31 && B * H < (int64_t(1) << 23);
}
bool prefill_fits(int64_t B, int64_t Tq, int64_t Tk, int32_t H) {
  return B >= 0 && B < (int64_t(1) << 24) && Tq >= 0 && Tq < k31 && Tk >= 0 && Tk < k31 - 64 &&
         (Tq / 64 + B) * H < (int64_t(1) << 23);
}

// The cache's sizes and pointers.
mx_status check_cache(const char* fn, int32_t kind, const void* k, const void* ks, const void* v, const void* vs,
                      int64_t pages, int32_t page_size, int32_t Hkv, int32_t D) {
  MX_CHECK(kind == MX_CACHE_MXFP8 || kind == MX_CACHE_BF16, "%s: unknown cache kind %d", fn, kind);
  MX_CHECK(page_fits(page_size), "%s: page_size = %d (a power of two, 16 to %d)", fn, page_size, MX_CACHE_MAX_PAGE);
  MX_CHECK(pages >= 1 && pages < k31, "%s: pages = %lld out of range", fn, (long long)pages);
  MX_CHECK(row_fits(Hkv, D), "%s: Hkv = %d, D = %d (D a multiple of %d up to 1024, Hkv * D up to 2^20)", fn, Hkv, D, MX_CACHE_BLOCK);
  MX_CHECK(pages * page_size * Hkv * D < (int64_t(1) << 46), "%s: %lld pages too large", fn, (long long)pages);
  MX_CHECK(k, "%s: null k_cache", fn);
  MX_CHECK(aligned(k, 16) && aligned(v, 16) && aligned(ks, 16) && aligned(vs, 16),
           "%s: caches and scales must be 16-byte aligned", fn);
  if (kind == MX_CACHE_MXFP8) {
    MX_CHECK(ks && (!v || vs), "%s: an MXFP8 cache needs its scales", fn);
  } else {
    MX_CHECK(!ks && !vs, "%s: a BF16 cache has no scales", fn);
  }
  MX_CHECK(v || !vs, "%s: v_scale without v_cache", fn);
  return MX_OK;
}

uint32_t shift_of(int32_t page_size) { return static_cast<uint32_t>(__builtin_ctz(static_cast<uint32_t>(page_size))); }

size_t cache_bytes(int32_t kind, int64_t pages, int32_t page_size, int32_t Hkv, int32_t D) {
  return static_cast<size_t>(pages) * page_size * Hkv * D * (kind == MX_CACHE_MXFP8 ? 1 : 2);
}
size_t scale_bytes(int32_t kind, int64_t pages, int32_t page_size, int32_t Hkv, int32_t D) {
  return kind == MX_CACHE_MXFP8 ? static_cast<size_t>(pages) * page_size * Hkv * (D / MX_CACHE_BLOCK) : 0;
}

KvCache view(const void* k, const uint8_t* ks, const void* v, const uint8_t* vs, int64_t pages, int32_t page_size,
             int32_t Hkv, const int32_t* table, int64_t max_pages) {
  KvCache c;
  c.k = static_cast<const uint8_t*>(k);
  c.ks = ks;
  c.v = v ? static_cast<const uint8_t*>(v) : c.k;      // a latent cache
  c.vs = v ? vs : ks;
  c.table = table;
  c.max_pages = static_cast<uint32_t>(max_pages);
  c.pages = static_cast<uint32_t>(pages);
  c.page_shift = shift_of(page_size);
  c.Hkv = static_cast<uint32_t>(Hkv);
  return c;
}

mx_status check_heads(const char* fn, int32_t H, int32_t Hkv, int32_t D, float scale) {
  MX_CHECK(head_dim(D), "%s: D = %d (64, 128, 256 or 512)", fn, D);
  MX_CHECK(heads_fit(H, Hkv), "%s: H = %d query heads over Hkv = %d key heads", fn, H, Hkv);
  // (the kernels multiply scores by scale * log2(e))
  MX_CHECK(scale > 0.0f && std::isfinite(scale * kLog2E), "%s: scale = %g (above 0, scale * log2(e) finite)", fn,
           static_cast<double>(scale));
  return MX_OK;
}

}  // namespace

extern "C" {

mx_status mx_kv_cache_write(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t T, int32_t Hkv,
                            int32_t D, const int64_t* slots, int32_t kind, void* k_cache, uint8_t* k_scale,
                            void* v_cache, uint8_t* v_scale, int64_t pages, int32_t page_size, void* stream) {
  const char* fn = "mx_kv_cache_write";
  const mx_status ok = check_cache(fn, kind, k_cache, k_scale, v_cache, v_scale, pages, page_size, Hkv, D);
  if (ok != MX_OK) return ok;
  const int64_t width = int64_t(Hkv) * D;
  MX_CHECK(T >= 0 && T < k31 && T * width < (int64_t(1) << 34), "%s: T = %lld rows of %lld out of range", fn,
           (long long)T, (long long)width);
  MX_CHECK((v != nullptr) == (v_cache != nullptr) || T == 0, "%s: v and v_cache go together (neither: a latent cache)", fn);
  if (T == 0) { clear_error(); return MX_OK; }
  MX_CHECK(k && slots, "%s: null tensor pointer", fn);
  MX_CHECK(k_stride >= width && k_stride % 8 == 0 && k_stride < k31 &&
               (!v || (v_stride >= width && v_stride % 8 == 0 && v_stride < k31)),
           "%s: strides %lld and %lld (multiples of 8, at least Hkv * D = %lld)", fn, (long long)k_stride,
           (long long)v_stride, (long long)width);
  MX_CHECK(aligned(k, 16) && aligned(v, 16) && aligned(slots, 8), "%s: k and v must be 16-byte, slots 8-byte aligned",
           fn);
  const size_t cb = cache_bytes(kind, pages, page_size, Hkv, D), sb = scale_bytes(kind, pages, page_size, Hkv, D);
  const Span part[] = {{"k_cache", k_cache, cb}, {"v_cache", v_cache, cb}, {"k_scale", k_scale, sb},
                       {"v_scale", v_scale, sb}, {"k", k, extent(T, k_stride, width)},
                       {"v", v, extent(T, v_stride, width)}, {"slots", slots, static_cast<size_t>(T) * 8}};
  const mx_status free = check_apart(fn, part, 4, 7);
  if (free != MX_OK) return free;
  MX_PREAMBLE();
  count(C_CACHE_WRITE);
  const mx_status st = launch_kv_write(k, k_stride, v, v_stride, T, Hkv, D, slots, kind == MX_CACHE_MXFP8, k_cache,
                                       k_scale, v_cache, v_scale, pages, shift_of(page_size),
                                       static_cast<hipStream_t>(stream));
  if (st == MX_OK) clear_error();
  return st;
}

mx_status mx_kv_cache_read(int32_t kind, const void* k_cache, const uint8_t* k_scale, const void* v_cache,
                           const uint8_t* v_scale, int64_t pages, int32_t page_size, int32_t Hkv, int32_t D,
                           const int32_t* block_table, int64_t B, int64_t max_pages, const int32_t* offsets,
                           int64_t rows, void* k, void* v, void* stream) {
  const char* fn = "mx_kv_cache_read";
  const mx_status ok = check_cache(fn, kind, k_cache, k_scale, v_cache, v_scale, pages, page_size, Hkv, D);
  if (ok != MX_OK) return ok;
  const int64_t width = int64_t(Hkv) * D;
  // (rows: 16 to a workgroup of 256, a launch has fewer than 2^32 threads)
  MX_CHECK(B >= 0 && B < k31 && rows >= 0 && rows <= (int64_t(1) << 28) - 16 && rows * width < (int64_t(1) << 34),
           "%s: B = %lld, rows = %lld of %lld out of range", fn, (long long)B, (long long)rows, (long long)width);
  MX_CHECK(max_pages >= 1 && max_pages < k31, "%s: max_pages = %lld out of range", fn, (long long)max_pages);
  MX_CHECK((v != nullptr) == (v_cache != nullptr) || rows == 0 || B == 0,
           "%s: v and v_cache go together (neither: a latent cache)", fn);
  if (B == 0 || rows == 0) { clear_error(); return MX_OK; }
  MX_CHECK(k && block_table && offsets, "%s: null tensor pointer", fn);
  MX_CHECK(aligned(k, 16) && aligned(v, 16) && aligned(block_table, 4) && aligned(offsets, 4),
           "%s: k and v must be 16-byte, block_table and offsets 4-byte aligned", fn);
  const size_t cb = cache_bytes(kind, pages, page_size, Hkv, D), sb = scale_bytes(kind, pages, page_size, Hkv, D);
  const size_t ob = static_cast<size_t>(rows) * width * 2;
  const Span part[] = {{"k", k, ob}, {"v", v, ob}, {"k_cache", k_cache, cb}, {"v_cache", v_cache, cb},
                       {"k_scale", k_scale, sb}, {"v_scale", v_scale, sb},
                       {"block_table", block_table, static_cast<size_t>(B) * max_pages * 4},
                       {"offsets", offsets, (static_cast<size_t>(B) + 1) * 4}};
  const mx_status free = check_apart(fn, part, 2, 8);
  if (free != MX_OK) return free;
  MX_PREAMBLE();
  count(C_CACHE_READ);
  const mx_status st = launch_kv_read(view(k_cache, k_scale, v_cache, v_scale, pages, page_size, Hkv, block_table, max_pages),
                                      kind == MX_CACHE_MXFP8, D, B, offsets, rows, k, v,
                                      static_cast<hipStream_t>(stream));
  if (st == MX_OK) clear_error();
  return st;
}

size_t mx_attn_decode_workspace_bytes(int64_t B, int32_t H, int32_t Hkv, int32_t D, int64_t max_pages,
                                      int32_t page_size) {
  if (B == 0 || !head_dim(D) || !heads_fit(H, Hkv) || !row_fits(Hkv, D) || !page_fits(page_size) ||
      !decode_fits(B, H, Hkv, max_pages, page_size))
    return 0;                                          // nothing to do, or sizes that a call refuses
  return decode_workspace_bytes(B, H, Hkv, D, max_pages * page_size);
}

mx_status mx_attn_decode(const void* q, int64_t q_stride, int64_t B, int32_t H, int32_t Hkv, int32_t D, int32_t kind,
                         const void* k_cache, const uint8_t* k_scale, const void* v_cache, const uint8_t* v_scale,
                         int64_t pages, int32_t page_size, const int32_t* block_table, int64_t max_pages,
                         const int32_t* lens, float scale, void* out, void* workspace, size_t workspace_bytes,
                         void* stream) {
  const char* fn = "mx_attn_decode";
  mx_status st = check_heads(fn, H, Hkv, D, scale);
  if (st != MX_OK) return st;
  st = check_cache(fn, kind, k_cache, k_scale, v_cache, v_scale, pages, page_size, Hkv, D);
  if (st != MX_OK) return st;
  MX_CHECK(decode_fits(B, H, Hkv, max_pages, page_size),
           "%s: B = %lld, H = %d, Hkv = %d, max_pages = %lld of %d tokens out of range", fn, (long long)B, H, Hkv,
           (long long)max_pages, page_size);
  if (B == 0) { clear_error(); return MX_OK; }
  MX_CHECK(q && block_table && lens && out, "%s: null tensor pointer", fn);
  MX_CHECK(q_stride >= int64_t(H) * D && q_stride % 8 == 0 && q_stride < k31,
           "%s: q_stride = %lld (a multiple of 8, at least H * D = %lld)", fn, (long long)q_stride, (long long)H * D);
  MX_CHECK(aligned(q, 16) && aligned(out, 16) && aligned(block_table, 4) && aligned(lens, 4),
           "%s: q and out must be 16-byte, block_table and lens 4-byte aligned", fn);
  const size_t need = mx_attn_decode_workspace_bytes(B, H, Hkv, D, max_pages, page_size);
  MX_CHECK(workspace && aligned(workspace, 16) && workspace_bytes >= need,
           "%s: workspace of %zu bytes (16-byte aligned) needed, got %zu", fn, need, workspace_bytes);
  const size_t cb = cache_bytes(kind, pages, page_size, Hkv, D), sb = scale_bytes(kind, pages, page_size, Hkv, D);
  const Span part[] = {{"out", out, static_cast<size_t>(B) * H * D * 2}, {"the workspace", workspace, need},
                       {"q", q, extent(B, q_stride, int64_t(H) * D)}, {"k_cache", k_cache, cb},
                       {"v_cache", v_cache, cb}, {"k_scale", k_scale, sb}, {"v_scale", v_scale, sb},
                       {"block_table", block_table, static_cast<size_t>(B) * max_pages * 4},
                       {"lens", lens, static_cast<size_t>(B) * 4}};
  st = check_apart(fn, part, 2, 9);
  if (st != MX_OK) return st;
  MX_PREAMBLE();
  count(C_ATTN_DECODE);
  st = launch_attn_decode(q, q_stride, B, H, D, kind == MX_CACHE_MXFP8,
                          view(k_cache, k_scale, v_cache, v_scale, pages, page_size, Hkv, block_table, max_pages), lens,
                          scale, out, workspace, static_cast<hipStream_t>(stream));
  if (st == MX_OK) clear_error();
  return st;
}

size_t mx_attn_prefill_workspace_bytes(int64_t B, int64_t Tq, int64_t Tk, int32_t H, int32_t Hkv, int32_t D) {
  if (B == 0 || Tq == 0 || !head_dim(D) || !heads_fit(H, Hkv) || !prefill_fits(B, Tq, Tk, H)) return 0;
  return prefill_workspace_bytes(B, Tq, Tk, H, Hkv, D);
}

mx_status mx_attn_prefill(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, const int32_t* q_offsets, const int32_t* k_offsets, int64_t B, int64_t Tq,
                          int64_t Tk, int32_t H, int32_t Hkv, int32_t D, float scale, void* out, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const char* fn = "mx_attn_prefill";
  mx_status st = check_heads(fn, H, Hkv, D, scale);
  if (st != MX_OK) return st;
  MX_CHECK(prefill_fits(B, Tq, Tk, H), "%s: B = %lld, Tq = %lld, Tk = %lld, H = %d out of range", fn, (long long)B,
           (long long)Tq, (long long)Tk, H);
  if (B == 0 || Tq == 0) { clear_error(); return MX_OK; }
  MX_CHECK(q && q_offsets && k_offsets && out && ((k && v) || Tk == 0), "%s: null tensor pointer", fn);
  const int64_t qw = int64_t(H) * D, kw = int64_t(Hkv) * D, most = int64_t(1) << 22;
  MX_CHECK(q_stride >= qw && q_stride % 8 == 0 && q_stride < k31, "%s: q_stride = %lld (a multiple of 8, at least H * D = %lld)",
           fn, (long long)q_stride, (long long)qw);
  MX_CHECK(Tk == 0 || (k_stride >= kw && k_stride % 8 == 0 && k_stride < most && v_stride >= kw && v_stride % 8 == 0 &&
                       v_stride < most),
           "%s: k_stride = %lld, v_stride = %lld (multiples of 8 below 2^22, at least Hkv * D = %lld)", fn,
           (long long)k_stride, (long long)v_stride, (long long)kw);
  MX_CHECK(aligned(q, 16) && aligned(k, 16) && aligned(v, 16) && aligned(out, 16) && aligned(q_offsets, 4) &&
               aligned(k_offsets, 4),
           "%s: q, k, v and out must be 16-byte, offsets 4-byte aligned", fn);
  const size_t need = mx_attn_prefill_workspace_bytes(B, Tq, Tk, H, Hkv, D);
  MX_CHECK(workspace_bytes >= need && (need == 0 || (workspace && aligned(workspace, 16))),
           "%s: workspace of %zu bytes (16-byte aligned) needed, got %zu", fn, need, workspace_bytes);
  const size_t offsets_bytes = (static_cast<size_t>(B) + 1) * 4;
  const Span part[] = {{"out", out, static_cast<size_t>(Tq) * qw * 2}, {"the workspace", workspace, need},
                       {"q", q, extent(Tq, q_stride, qw)}, {"k", k, extent(Tk, k_stride, kw)},
                       {"v", v, extent(Tk, v_stride, kw)}, {"q_offsets", q_offsets, offsets_bytes},
                       {"k_offsets", k_offsets, offsets_bytes}};
  st = check_apart(fn, part, 2, 7);
  if (st != MX_OK) return st;
  MX_PREAMBLE();
  count(C_ATTN_PREFILL);
  st = launch_attn_prefill(q, q_stride, k, k_stride, v, v_stride, q_offsets, k_offsets, B, Tq, Tk, H, Hkv, D, scale,
                           out, workspace, static_cast<hipStream_t>(stream));
  if (st == MX_OK) clear_error();
  return st;
}

}  // extern "C"
