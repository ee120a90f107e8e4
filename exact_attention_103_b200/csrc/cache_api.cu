// cache_api.cu -- the C ABI of the serving operators (declared in
// include/attn_cache.h): argument checks and launches.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "attn_internal.h"
#include "cache_ops.h"

using attn_internal::report;

namespace {

attn_status_t fail(attn_status_t s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
attn_status_t fail(attn_status_t s, const char* fmt, ...) {
  char text[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  return report(s, text);
}

attn_status_t launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? ATTN_OK : fail(ATTN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

using attn::kMaxSequences;
constexpr int kMaxRequests = 8192;  // slots, and requests of one alloc or fork (shared-memory lists)
constexpr int kMaxMask = 256;

attn_status_t check_cache(const attn_cache_t* c) {
  if (!c) return fail(ATTN_ERR_INVALID_ARG, "cache is null");
  if (c->layers <= 0 || c->pages <= 0 || c->heads <= 0 || c->slots <= 0 || c->max_pages <= 0)
    return fail(ATTN_ERR_INVALID_ARG, "cache: layers=%d pages=%d heads=%d slots=%d max_pages=%d", c->layers, c->pages,
                c->heads, c->slots, c->max_pages);
  if (c->d != 64 && c->d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim %d (supported: 64, 128)", c->d);
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
    return fail(ATTN_ERR_UNSUPPORTED, "page size %d (supported: powers of two from 16 to 1024)", c->page_size);
  if (c->slots > kMaxRequests) return fail(ATTN_ERR_UNSUPPORTED, "cache: %d slots (at most %d)", c->slots, kMaxRequests);
  // grid dimensions, 32-bit row coordinates of the tensor maps, 32-bit token positions
  if (c->layers > 4096 || c->heads > 1024 ||
      static_cast<int64_t>(c->layers) * c->pages * c->page_size > INT32_MAX - 2048 ||
      static_cast<int64_t>(c->max_pages) * c->page_size > INT32_MAX - 2048)
    return fail(ATTN_ERR_UNSUPPORTED, "cache too large for 32-bit row indexing");
  if (!c->k || !c->v || !c->page_table || !c->lens || !c->refs)
    return fail(ATTN_ERR_INVALID_ARG, "cache: null pointer");
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4) || !aligned(c->lens, 4) ||
      !aligned(c->refs, 4))
    return fail(ATTN_ERR_INVALID_ARG, "cache: k and v must be 16-byte aligned, tables 4-byte");
  if (c->e4m3 != 0 && c->e4m3 != 1) return fail(ATTN_ERR_INVALID_ARG, "cache: e4m3 must be 0 or 1");
  if (!(std::isfinite(c->k_scale) && c->k_scale > 0.f && std::isfinite(c->v_scale) && c->v_scale > 0.f))
    return fail(ATTN_ERR_INVALID_ARG, "cache scales must be finite and > 0");
  return ATTN_OK;
}

attn_status_t check_list(const void* p, const char* name) {
  if (!p) return fail(ATTN_ERR_INVALID_ARG, "%s is null", name);
  if (!aligned(p, 4)) return fail(ATTN_ERR_INVALID_ARG, "%s must be 4-byte aligned", name);
  return ATTN_OK;
}

attn_status_t check_plan(const attn_rope_plan_t* p, int d) {
  if (!p || !p->turns) return fail(ATTN_ERR_INVALID_ARG, "rotary plan is null");
  if (!aligned(p->turns, 8)) return fail(ATTN_ERR_INVALID_ARG, "rotary plan must be 8-byte aligned");
  if (p->dim <= 0 || p->dim % 16 || p->dim > d)
    return fail(ATTN_ERR_UNSUPPORTED, "%d rotated values (supported: multiples of 16 up to the head dim %d)", p->dim, d);
  if (!(std::isfinite(p->amplitude) && p->amplitude > 0.f))
    return fail(ATTN_ERR_INVALID_ARG, "rotary amplitude must be finite and > 0");
  return ATTN_OK;
}

// Rows of a tensor: 16-byte accesses at every stride.
attn_status_t check_rows(const attn_rows_t& t, const char* name, bool batch, bool dst, int size) {
  if (t.heads <= 0 || t.heads > 65536) return fail(ATTN_ERR_INVALID_ARG, "%s: %d heads", name, t.heads);
  if (!t.src || (dst && !t.dst)) return fail(ATTN_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!aligned(t.src, 16) || (dst && !aligned(t.dst, 16)))
    return fail(ATTN_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  const int64_t unit = 16 / size;
  const int64_t strides[6] = {t.src_token, t.src_head, batch ? t.src_batch : 0, dst ? t.dst_token : 0,
                              dst ? t.dst_head : 0, dst && batch ? t.dst_batch : 0};
  for (int64_t s : strides)
    if (s % unit) return fail(ATTN_ERR_INVALID_ARG, "%s: strides must be multiples of 16 bytes", name);
  return ATTN_OK;
}

attn_status_t device(int** err, int* sms) { return attn_internal::prepare_device(err, sms); }

cudaStream_t cu(attn_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

#define ATTN_TRY(x)                       \
  do {                                    \
    const attn_status_t try_st = (x);     \
    if (try_st != ATTN_OK) return try_st; \
  } while (0)

}  // namespace

extern "C" {

attn_status_t attn_rope(const attn_rope_plan_t* plan, int inverse, attn_type_t type, const attn_rows_t* tensors,
                        int count, int d, int B, int N, const int32_t* cu_seqlens, const int32_t* positions,
                        attn_stream_t stream) {
  if (B < 0 || N < 0) return fail(ATTN_ERR_INVALID_ARG, "B=%d N=%d", B, N);
  if (type != ATTN_BF16 && type != ATTN_FP16 && type != ATTN_FP32)
    return fail(ATTN_ERR_UNSUPPORTED, "type %d (supported: bf16, fp16, fp32)", static_cast<int>(type));
  if (d <= 0 || d % 16 || d > 256) return fail(ATTN_ERR_UNSUPPORTED, "head dim %d (supported: multiples of 16 up to 256)", d);
  ATTN_TRY(check_plan(plan, d));
  if (count != 1 && count != 2) return fail(ATTN_ERR_INVALID_ARG, "%d tensors (1 or 2)", count);
  if (!tensors) return fail(ATTN_ERR_INVALID_ARG, "tensors is null");
  if (cu_seqlens) {
    if (B > kMaxSequences) return fail(ATTN_ERR_UNSUPPORTED, "packed batches hold at most %d sequences", kMaxSequences);
    ATTN_TRY(check_list(cu_seqlens, "cu_seqlens"));
  }
  if (positions) ATTN_TRY(check_list(positions, "positions"));
  // a packed batch of no sequence has no token to turn, unless positions name each token's
  if (N == 0 || (B == 0 && !(cu_seqlens && positions))) return ATTN_OK;
  for (int i = 0; i < count; ++i)
    ATTN_TRY(check_rows(tensors[i], i ? "k" : "q", !cu_seqlens, true, type == ATTN_FP32 ? 4 : 2));
  const int64_t tokens = cu_seqlens ? N : static_cast<int64_t>(B) * N;
  if (tokens > INT32_MAX - kMaxSequences) return fail(ATTN_ERR_UNSUPPORTED, "too many tokens for 32-bit indexing");
  attn::RopeArgs a = {};
  a.plan = *plan;
  a.t[0] = tensors[0];
  if (count > 1) a.t[1] = tensors[1];
  a.inverse = inverse;
  a.d = d;
  a.B = B;
  a.N = N;
  a.tokens = static_cast<int>(tokens);
  a.cu = cu_seqlens;
  a.positions = positions;
  int sms = 0;
  ATTN_TRY(device(&a.err, &sms));
  return launched(attn::launch_rope(a, type, sms, cu(stream)), "rotary kernel launch");
}

attn_status_t attn_rope_append(const attn_cache_t* cache, int layer, const attn_rope_plan_t* plan,
                               const attn_rows_t* q, const attn_rows_t* k, const attn_rows_t* v, int B, int T,
                               const int32_t* cu_q, const int32_t* slots, const int32_t* positions,
                               attn_stream_t stream) {
  ATTN_TRY(check_cache(cache));
  if (layer < 0 || layer >= cache->layers) return fail(ATTN_ERR_INVALID_ARG, "layer %d of %d", layer, cache->layers);
  if (B < 0 || T < 0) return fail(ATTN_ERR_INVALID_ARG, "B=%d T=%d", B, T);
  if (B > kMaxSequences) return fail(ATTN_ERR_UNSUPPORTED, "at most %d sequences", kMaxSequences);
  if (plan) ATTN_TRY(check_plan(plan, cache->d));
  if (!slots && B > cache->slots) return fail(ATTN_ERR_INVALID_ARG, "%d sequences for %d slots", B, cache->slots);
  if (B == 0 || T == 0) return ATTN_OK;
  if (T > INT32_MAX - kMaxSequences) return fail(ATTN_ERR_UNSUPPORTED, "too many tokens for 32-bit indexing");
  ATTN_TRY(check_list(cu_q, "cu_q"));
  if (slots) ATTN_TRY(check_list(slots, "slots"));
  if (positions) ATTN_TRY(check_list(positions, "positions"));
  if (!k || !v) return fail(ATTN_ERR_INVALID_ARG, "k or v is null");
  if (q) ATTN_TRY(check_rows(*q, "q", false, true, 2));
  ATTN_TRY(check_rows(*k, "k", false, false, 2));
  ATTN_TRY(check_rows(*v, "v", false, false, 2));
  if (k->heads != cache->heads || v->heads != cache->heads)
    return fail(ATTN_ERR_INVALID_ARG, "k and v must have the cache's %d heads", cache->heads);
  attn::RopeArgs a = {};
  if (plan) a.plan = *plan;
  if (q) a.t[0] = *q;
  a.t[1] = *k;
  a.t[2] = *v;
  a.d = cache->d;
  a.B = B;
  a.N = T;
  a.tokens = T;
  a.cu = cu_q;
  a.positions = positions;
  a.cache = *cache;
  a.layer = layer;
  a.slots = slots;
  int sms = 0;
  ATTN_TRY(device(&a.err, &sms));
  return launched(attn::launch_append(a, sms, cu(stream)), "append kernel launch");
}

attn_status_t attn_cache_alloc(const attn_cache_t* cache, const int32_t* slots, const int32_t* new_lens, int n,
                               int32_t* granted, attn_stream_t stream) {
  ATTN_TRY(check_cache(cache));
  if (n < 0 || n > kMaxRequests) return fail(ATTN_ERR_INVALID_ARG, "%d requests (at most %d)", n, kMaxRequests);
  if (n == 0) return ATTN_OK;
  ATTN_TRY(check_list(slots, "slots"));
  ATTN_TRY(check_list(new_lens, "new_lens"));
  ATTN_TRY(check_list(granted, "granted"));
  int *err = nullptr, sms = 0;
  ATTN_TRY(device(&err, &sms));
  return launched(attn::launch_alloc(*cache, slots, new_lens, n, granted, err, cu(stream)), "alloc kernel launch");
}

attn_status_t attn_cache_free(const attn_cache_t* cache, const int32_t* slots, int n, attn_stream_t stream) {
  ATTN_TRY(check_cache(cache));
  if (n < 0) return fail(ATTN_ERR_INVALID_ARG, "%d slots", n);
  if (n == 0) return ATTN_OK;
  ATTN_TRY(check_list(slots, "slots"));
  int *err = nullptr, sms = 0;
  ATTN_TRY(device(&err, &sms));
  return launched(attn::launch_free(*cache, slots, n, err, cu(stream)), "free kernel launch");
}

size_t attn_cache_fork_workspace_size(int n) { return n > 0 ? static_cast<size_t>(n) * 16 : 0; }

attn_status_t attn_cache_fork(const attn_cache_t* cache, const int32_t* src, const int32_t* dst, int n,
                              int32_t* granted, void* workspace, size_t workspace_bytes, attn_stream_t stream) {
  ATTN_TRY(check_cache(cache));
  if (n < 0 || n > kMaxRequests) return fail(ATTN_ERR_INVALID_ARG, "%d requests (at most %d)", n, kMaxRequests);
  if (n == 0) return ATTN_OK;
  ATTN_TRY(check_list(src, "src"));
  ATTN_TRY(check_list(dst, "dst"));
  ATTN_TRY(check_list(granted, "granted"));
  const size_t need = attn_cache_fork_workspace_size(n);
  if (workspace_bytes < need || !workspace || !aligned(workspace, 16))
    return fail(ATTN_ERR_WORKSPACE, "workspace of %zu bytes (16-byte aligned) needed", need);
  int *err = nullptr, sms = 0;
  ATTN_TRY(device(&err, &sms));
  return launched(attn::launch_fork(*cache, src, dst, n, granted, workspace, err, cu(stream)), "fork kernel launch");
}

attn_status_t attn_cache_copy(const attn_cache_t* cache, const int32_t* src, const int32_t* dst, int n,
                              attn_stream_t stream) {
  ATTN_TRY(check_cache(cache));
  if (n < 0) return fail(ATTN_ERR_INVALID_ARG, "%d copies", n);
  if (n == 0) return ATTN_OK;
  ATTN_TRY(check_list(src, "src"));
  ATTN_TRY(check_list(dst, "dst"));
  int *err = nullptr, sms = 0;
  ATTN_TRY(device(&err, &sms));
  return launched(attn::launch_copy(*cache, src, dst, n, err, cu(stream)), "copy kernel launch");
}

attn_status_t attn_cache_compact(const attn_cache_t* cache, const int32_t* cu_q, const int32_t* path, int path_width,
                                 const int32_t* accepted, const int32_t* slots, int B, attn_stream_t stream) {
  ATTN_TRY(check_cache(cache));
  if (B < 0 || path_width < 0) return fail(ATTN_ERR_INVALID_ARG, "B=%d path_width=%d", B, path_width);
  if (B > kMaxSequences) return fail(ATTN_ERR_UNSUPPORTED, "at most %d sequences", kMaxSequences);
  if (!slots && B > cache->slots) return fail(ATTN_ERR_INVALID_ARG, "%d sequences for %d slots", B, cache->slots);
  if (B == 0) return ATTN_OK;
  ATTN_TRY(check_list(cu_q, "cu_q"));
  if (path_width > 0) ATTN_TRY(check_list(path, "path"));
  ATTN_TRY(check_list(accepted, "accepted"));
  if (slots) ATTN_TRY(check_list(slots, "slots"));
  int *err = nullptr, sms = 0;
  ATTN_TRY(device(&err, &sms));
  return launched(attn::launch_compact(*cache, cu_q, path, path_width, accepted, slots, B, err, cu(stream)),
                  "compact kernel launch");
}

size_t attn_tree_workspace_size(int d) { return d == 64 || d == 128 ? attn::tree_workspace(d) : 0; }

attn_status_t attn_tree_fwd(const attn_cache_t* cache, int layer, const void* q, void* o, float* lse, int Hq, int B,
                            int T, const int32_t* cu_q, const int32_t* slots, const uint8_t* mask, int mask_width,
                            float scale, void* workspace, size_t workspace_bytes, attn_stream_t stream) {
  ATTN_TRY(check_cache(cache));
  if (layer < 0 || layer >= cache->layers) return fail(ATTN_ERR_INVALID_ARG, "layer %d of %d", layer, cache->layers);
  if (B < 0 || T < 0) return fail(ATTN_ERR_INVALID_ARG, "B=%d T=%d", B, T);
  if (Hq <= 0 || Hq % cache->heads || Hq / cache->heads > 128)
    return fail(ATTN_ERR_UNSUPPORTED, "%d query heads over %d cache heads (a multiple, up to 128 times)", Hq, cache->heads);
  if (B > kMaxSequences) return fail(ATTN_ERR_UNSUPPORTED, "at most %d sequences", kMaxSequences);
  if (!slots && B > cache->slots) return fail(ATTN_ERR_INVALID_ARG, "%d sequences for %d slots", B, cache->slots);
  if (!(std::isfinite(scale) && scale > 0.f)) return fail(ATTN_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (mask && (mask_width <= 0 || mask_width > kMaxMask))
    return fail(ATTN_ERR_UNSUPPORTED, "mask width %d (1 to %d)", mask_width, kMaxMask);
  if (B == 0 || T == 0) return ATTN_OK;
  if (!q || !o || !lse) return fail(ATTN_ERR_INVALID_ARG, "null tensor pointer");
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4))
    return fail(ATTN_ERR_INVALID_ARG, "q/o must be 16-byte aligned and lse 4-byte aligned");
  ATTN_TRY(check_list(cu_q, "cu_q"));
  if (slots) ATTN_TRY(check_list(slots, "slots"));
  if (static_cast<int64_t>(T) * Hq > INT32_MAX - 2048)
    return fail(ATTN_ERR_UNSUPPORTED, "too many query rows for 32-bit indexing");
  const size_t need = attn_tree_workspace_size(cache->d);
  if (workspace_bytes < need || (need > 0 && (!workspace || !aligned(workspace, 256))))
    return fail(ATTN_ERR_WORKSPACE, "workspace of %zu bytes (256-byte aligned) needed", need);
  attn::TreeArgs a = {};
  a.cache = *cache;
  a.layer = layer;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.Hq = Hq;
  a.B = B;
  a.T = T;
  a.cu = cu_q;
  a.slots = slots;
  a.mask = mask;
  a.mask_width = mask_width;
  a.scale = scale;
  a.ws = workspace;
  int sms = 0;
  ATTN_TRY(device(&a.err, &sms));
  cudaError_t e = cudaSuccess;
  const attn_status_t st = attn::launch_tree(a, sms, cu(stream), &e);
  if (st == ATTN_ERR_UNSUPPORTED) return fail(st, "problem too large for 32-bit tile indexing");
  if (st != ATTN_OK) return fail(st, "cuTensorMapEncodeTiled rejected the q/k/v views");
  return launched(e, "attention kernel launch");
}

}  // extern "C"
