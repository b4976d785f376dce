// kvc_paged.cu -- validating C-ABI layer of the paged cache: kvc_page_plan,
// kvc_page_write and kvc_paged_attention.  As in kvc_host.cu, every argument
// the host can check is checked before anything is launched.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "kvc_paged_internal.h"

namespace kvc {
namespace {

kvc_status fail(kvc_status st, const char* fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return set_last_error(st, msg);
}

kvc_status cuda_fail(cudaError_t e, const char* what) {
  return fail(KVC_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

#define KVC_TRY(expr)                    \
  do {                                   \
    const kvc_status _st = (expr);       \
    if (_st != KVC_OK) return _st;       \
  } while (0)

int64_t elem_bytes(kvc_dtype t) { return t == KVC_BF16 ? 2 : 4; }

// Byte range [lo, hi) of device memory.
struct Span {
  uintptr_t lo, hi;
};

Span span(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Span{lo, lo + static_cast<uintptr_t>(bytes)};
}

bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

kvc_status check_ptr(const void* p, const char* name, unsigned align) {
  if (p == nullptr) return fail(KVC_ERR_INVALID_ARGUMENT, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & (align - 1))
    return fail(KVC_ERR_ALIGNMENT, "%s must be %u-byte aligned", name, align);
  return KVC_OK;
}

kvc_status check_paged(const kvc_paged* pg) {
  if (pg == nullptr) return fail(KVC_ERR_INVALID_ARGUMENT, "paged descriptor is NULL");
  if (pg->dtype != KVC_BF16 && pg->dtype != KVC_F32)
    return fail(KVC_ERR_DTYPE, "unknown dtype %d", static_cast<int>(pg->dtype));
  if (pg->n_pages < 1 || pg->page_size < 1 || pg->L < 1 || pg->H < 1 || pg->max_blocks < 1)
    return fail(KVC_ERR_SHAPE,
                "n_pages, page_size, L, H, max_blocks must be >= 1 (got %d, %d, %d, %d, %d)",
                pg->n_pages, pg->page_size, pg->L, pg->H, pg->max_blocks);
  if (pg->R < 0) return fail(KVC_ERR_SHAPE, "R = %d < 0", pg->R);
  if (pg->n_pages > (1 << 30))
    return fail(KVC_ERR_UNSUPPORTED, "n_pages = %d exceeds 2^30", pg->n_pages);
  if (static_cast<int64_t>(pg->max_blocks) * pg->page_size > (int64_t(1) << 30))
    return fail(KVC_ERR_UNSUPPORTED, "max_blocks * page_size = %lld exceeds 2^30 tokens",
                static_cast<long long>(pg->max_blocks) * pg->page_size);
  return KVC_OK;
}

kvc_status check_head_dim(const kvc_paged* pg) {
  if (pg->dtype == KVC_BF16) {
    if (pg->d != 64 && pg->d != 128)
      return fail(KVC_ERR_UNSUPPORTED, "bf16 head dim must be 64 or 128 (got %d)", pg->d);
  } else if (pg->d < 4 || pg->d > 256 || (pg->d % 4) != 0) {
    return fail(KVC_ERR_UNSUPPORTED, "f32 head dim must be a multiple of 4 in [4, 256] (got %d)",
                pg->d);
  }
  return KVC_OK;
}

kvc_status check_view(const kvc_paged* pg, const kvc_cache_view& v, const char* name) {
  if (v.base == nullptr) return fail(KVC_ERR_INVALID_ARGUMENT, "%s.base is NULL", name);
  if (v.s_req < 0 || v.s_layer < 0 || v.s_head < 0 || v.s_tok < pg->d)
    return fail(KVC_ERR_SHAPE, "%s: strides must be >= 0 and s_tok >= d", name);
  const int64_t e = elem_bytes(pg->dtype), lim = (int64_t(1) << 40) / e;
  if (v.s_req >= lim || v.s_layer >= lim || v.s_head >= lim || v.s_tok >= lim)
    return fail(KVC_ERR_UNSUPPORTED, "%s: byte strides must be < 2^40", name);
  if ((reinterpret_cast<uintptr_t>(v.base) & 15) || (v.s_req * e) % 16 || (v.s_layer * e) % 16 ||
      (v.s_head * e) % 16 || (v.s_tok * e) % 16)
    return fail(KVC_ERR_ALIGNMENT, "%s: base and byte strides must be multiples of 16", name);
  return KVC_OK;
}

kvc_status check_pool(const kvc_paged* pg, const kvc_cache_view& v, const char* name) {
  KVC_TRY(check_view(pg, v, name));
  if ((pg->n_pages > 1 && v.s_req < pg->d) || (pg->L > 1 && v.s_layer < pg->d) ||
      (pg->H > 1 && v.s_head < pg->d))
    return fail(KVC_ERR_SHAPE, "%s: strides of a pool must be >= d", name);
  return KVC_OK;
}

Span view_span(const kvc_paged* pg, const kvc_cache_view& v, int64_t R, int64_t L, int64_t T) {
  const int64_t last = (R - 1) * v.s_req + (L - 1) * v.s_layer + (pg->H - 1) * v.s_head +
                       (T - 1) * v.s_tok + pg->d;
  return span(v.base, last * elem_bytes(pg->dtype));
}

kvc_status check_attn(const kvc_paged* pg, const kvc_attn_params* at) {
  if (at == nullptr) return fail(KVC_ERR_INVALID_ARGUMENT, "attention descriptor is NULL");
  if (at->n_q_heads < 1 || at->n_q_heads % pg->H != 0)
    return fail(KVC_ERR_SHAPE, "n_q_heads = %d is no multiple of H = %d", at->n_q_heads, pg->H);
  if (at->n_q_heads / pg->H > 64)
    return fail(KVC_ERR_UNSUPPORTED, "n_q_heads / H = %d exceeds 64", at->n_q_heads / pg->H);
  if (at->n_tokens < 0 || at->n_tokens > (1 << 30))
    return fail(KVC_ERR_SHAPE, "n_tokens = %d outside [0, 2^30]", at->n_tokens);
  if (at->layer < 0 || at->layer >= pg->L)
    return fail(KVC_ERR_SHAPE, "layer %d outside [0, %d)", at->layer, pg->L);
  if (at->causal != 0 && at->causal != 1)
    return fail(KVC_ERR_INVALID_ARGUMENT, "causal = %d is neither 0 nor 1", at->causal);
  if (at->window < 0) return fail(KVC_ERR_INVALID_ARGUMENT, "window = %d < 0", at->window);
  if (at->window > 0 && !at->causal)
    return fail(KVC_ERR_INVALID_ARGUMENT, "a window needs causal = 1");
  if (!(at->scale > 0.0f) || !std::isfinite(at->scale))
    return fail(KVC_ERR_INVALID_ARGUMENT, "scale must be finite and > 0");
  return KVC_OK;
}

// Rows [N, Hq, d] with element strides.
kvc_status check_rows(const kvc_paged* pg, const kvc_attn_params* at, const void* p, int64_t s_tok,
                      int64_t s_head, const char* name) {
  KVC_TRY(check_ptr(p, name, 16));
  const int64_t e = elem_bytes(pg->dtype), lim = (int64_t(1) << 40) / e;
  if (s_tok < 0 || s_head < 0 || (at->n_q_heads > 1 && s_head < pg->d) ||
      (at->n_tokens > 1 && s_tok < pg->d))
    return fail(KVC_ERR_SHAPE, "%s: strides must be >= d", name);
  if (s_tok >= lim || s_head >= lim)
    return fail(KVC_ERR_UNSUPPORTED, "%s: byte strides must be < 2^40", name);
  if ((s_tok * e) % 16 || (s_head * e) % 16)
    return fail(KVC_ERR_ALIGNMENT, "%s: byte strides must be multiples of 16", name);
  return KVC_OK;
}

Span rows_span(const kvc_paged* pg, const kvc_attn_params* at, const void* p, int64_t s_tok,
               int64_t s_head) {
  const int64_t last =
      (at->n_tokens - 1) * s_tok + (at->n_q_heads - 1) * s_head + pg->d;
  return span(p, last * elem_bytes(pg->dtype));
}

size_t attn_workspace_bytes(const kvc_paged* pg) {
  return pg->dtype == KVC_BF16 ? attn_tc_workspace_bytes(pg->d) : attn_f32_workspace_bytes(pg->d);
}

}  // namespace
}  // namespace kvc

using namespace kvc;

extern "C" {

kvc_status kvc_page_plan(const kvc_paged* pg, const int32_t* new_lens, const int32_t* kv_lens,
                         int32_t* kv_lens_out, int32_t* block_table, int32_t* free_pages,
                         const int32_t* n_free, int32_t* n_free_out, int32_t max_tokens,
                         int32_t* q_start, int64_t* slot_map, int32_t* positions,
                         int32_t* plan_status, cudaStream_t stream) {
  KVC_TRY(check_paged(pg));
  if (pg->R > kMaxPlanRequests)
    return fail(KVC_ERR_UNSUPPORTED, "R = %d exceeds %d requests per plan", pg->R,
                kMaxPlanRequests);
  if (max_tokens < 0 || max_tokens > (1 << 30))
    return fail(KVC_ERR_SHAPE, "max_tokens = %d outside [0, 2^30]", max_tokens);
  if (pg->R > 0) {
    KVC_TRY(check_ptr(new_lens, "new_lens", 4));
    KVC_TRY(check_ptr(kv_lens, "kv_lens", 4));
    KVC_TRY(check_ptr(kv_lens_out, "kv_lens_out", 4));
    KVC_TRY(check_ptr(block_table, "block_table", 4));
    KVC_TRY(check_ptr(plan_status, "plan_status", 4));
  }
  KVC_TRY(check_ptr(free_pages, "free_pages", 4));
  KVC_TRY(check_ptr(n_free, "n_free", 4));
  KVC_TRY(check_ptr(n_free_out, "n_free_out", 4));
  KVC_TRY(check_ptr(q_start, "q_start", 4));
  if (max_tokens > 0) {
    KVC_TRY(check_ptr(slot_map, "slot_map", 8));
    KVC_TRY(check_ptr(positions, "positions", 4));
  }
  const int64_t R = pg->R;
  const struct {
    Span s;
    const char* name;
    bool written;
  } buf[] = {{span(new_lens, 4 * R), "new_lens", false},
             {span(kv_lens, 4 * R), "kv_lens", false},
             {span(n_free, 4), "n_free", false},
             {span(block_table, 4 * R * pg->max_blocks), "block_table", true},
             {span(free_pages, 4 * int64_t(pg->n_pages)), "free_pages", true},
             {span(kv_lens_out, 4 * R), "kv_lens_out", true},
             {span(n_free_out, 4), "n_free_out", true},
             {span(q_start, 4 * (R + 1)), "q_start", true},
             {span(slot_map, 8 * int64_t(max_tokens)), "slot_map", true},
             {span(positions, 4 * int64_t(max_tokens)), "positions", true},
             {span(plan_status, 4 * R), "plan_status", true}};
  const int n = static_cast<int>(sizeof(buf) / sizeof(buf[0]));
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if ((buf[i].written || buf[j].written) && overlap(buf[i].s, buf[j].s))
        return fail(KVC_ERR_ALIAS, "%s and %s overlap", buf[i].name, buf[j].name);
  PlanArgs a{};
  a.new_lens = new_lens;
  a.kv_in = kv_lens;
  a.kv_out = kv_lens_out;
  a.table = block_table;
  a.free_pages = free_pages;
  a.n_free_in = n_free;
  a.n_free_out = n_free_out;
  a.q_start = q_start;
  a.slots = slot_map;
  a.positions = positions;
  a.status = plan_status;
  a.R = pg->R;
  a.P = pg->n_pages;
  a.B = pg->page_size;
  a.width = pg->max_blocks;
  a.max_tokens = max_tokens;
  const cudaError_t e = launch_page_plan(a, stream);
  if (e != cudaSuccess) return cuda_fail(e, "kvc_page_plan launch");
  return KVC_OK;
}

kvc_status kvc_page_write(const kvc_paged* pg, int32_t n_src, int32_t T, int32_t layer,
                          int32_t n_layers, kvc_cache_view src_K, kvc_cache_view src_V,
                          const int64_t* slot_map, kvc_cache_view pool_K, kvc_cache_view pool_V,
                          cudaStream_t stream) {
  KVC_TRY(check_paged(pg));
  KVC_TRY(check_head_dim(pg));
  if (n_src < 0 || T < 0)
    return fail(KVC_ERR_SHAPE, "n_src and T must be >= 0 (got %d, %d)", n_src, T);
  if (n_layers < 1 || layer < 0 || static_cast<int64_t>(layer) + n_layers > pg->L)
    return fail(KVC_ERR_SHAPE, "layers [%d, %lld) outside [0, %d)", layer,
                static_cast<long long>(layer) + n_layers, pg->L);
  if (static_cast<int64_t>(n_layers) * pg->H > 65535)
    return fail(KVC_ERR_UNSUPPORTED, "n_layers * H = %lld exceeds 65535",
                static_cast<long long>(n_layers) * pg->H);
  KVC_TRY(check_pool(pg, pool_K, "pool_K"));
  KVC_TRY(check_pool(pg, pool_V, "pool_V"));
  if (n_src == 0 || T == 0) return KVC_OK;           // sources of no rows may have no address
  KVC_TRY(check_view(pg, src_K, "src_K"));
  KVC_TRY(check_view(pg, src_V, "src_V"));
  KVC_TRY(check_ptr(slot_map, "slot_map", 8));
  const Span pools[2] = {view_span(pg, pool_K, pg->n_pages, pg->L, pg->page_size),
                         view_span(pg, pool_V, pg->n_pages, pg->L, pg->page_size)};
  for (const Span& p : pools) {
    if (overlap(p, view_span(pg, src_K, n_src, n_layers, T)) ||
        overlap(p, view_span(pg, src_V, n_src, n_layers, T)))
      return fail(KVC_ERR_ALIAS, "src_K/src_V may not overlap pool_K/pool_V");
    if (overlap(p, span(slot_map, 8 * int64_t(n_src) * T)))
      return fail(KVC_ERR_ALIAS, "slot_map may not overlap pool_K/pool_V");
  }
  WriteArgs a{};
  a.src[0] = to_view(src_K);
  a.src[1] = to_view(src_V);
  a.pool[0] = to_view(pool_K);
  a.pool[1] = to_view(pool_V);
  a.slots = slot_map;
  a.rows = static_cast<int64_t>(n_src) * T;
  a.n_slots = static_cast<int64_t>(pg->n_pages) * pg->page_size;
  a.T = T;
  a.B = pg->page_size;
  a.L0 = layer;
  a.nl = n_layers;
  a.H = pg->H;
  a.elem = static_cast<int32_t>(elem_bytes(pg->dtype));
  a.vec_row = pg->d * a.elem / 16;
  const cudaError_t e = launch_page_write(a, stream);
  if (e != cudaSuccess) return cuda_fail(e, "kvc_page_write launch");
  return KVC_OK;
}

size_t kvc_paged_attention_workspace(const kvc_paged* pg, const kvc_attn_params* at) {
  if (check_paged(pg) != KVC_OK || check_head_dim(pg) != KVC_OK || check_attn(pg, at) != KVC_OK)
    return 0;
  return attn_workspace_bytes(pg);
}

kvc_status kvc_paged_attention(const kvc_paged* pg, const kvc_attn_params* at, const void* q,
                               kvc_cache_view pool_K, kvc_cache_view pool_V,
                               const int32_t* block_table, const int32_t* q_start,
                               const int32_t* kv_lens, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, int32_t* dev_status, cudaStream_t stream) {
  KVC_TRY(check_paged(pg));
  KVC_TRY(check_head_dim(pg));
  KVC_TRY(check_attn(pg, at));
  KVC_TRY(check_pool(pg, pool_K, "pool_K"));
  KVC_TRY(check_pool(pg, pool_V, "pool_V"));
  if (at->n_tokens > 0) {
    if (pg->R > 0) {
      KVC_TRY(check_ptr(block_table, "block_table", 4));
      KVC_TRY(check_ptr(q_start, "q_start", 4));
      KVC_TRY(check_ptr(kv_lens, "kv_lens", 4));
    }
    KVC_TRY(check_rows(pg, at, q, at->q_s_tok, at->q_s_head, "q"));
    KVC_TRY(check_rows(pg, at, out, at->out_s_tok, at->out_s_head, "out"));
  }
  if (reinterpret_cast<uintptr_t>(lse) & 3)
    return fail(KVC_ERR_ALIGNMENT, "lse must be 4-byte aligned");
  KVC_TRY(check_ptr(dev_status, "dev_status", 4));
  const size_t bytes = attn_workspace_bytes(pg);
  if (workspace == nullptr || workspace_bytes < bytes)
    return fail(KVC_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", bytes,
                workspace == nullptr ? size_t(0) : workspace_bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(KVC_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  if (at->n_tokens == 0 || pg->R == 0) return KVC_OK;
  const Span o = rows_span(pg, at, out, at->out_s_tok, at->out_s_head);
  const Span s = span(lse, lse == nullptr ? 0 : 4 * int64_t(at->n_tokens) * at->n_q_heads);
  const Span ws = span(workspace, static_cast<int64_t>(bytes));
  const Span in[] = {rows_span(pg, at, q, at->q_s_tok, at->q_s_head),
                     view_span(pg, pool_K, pg->n_pages, pg->L, pg->page_size),
                     view_span(pg, pool_V, pg->n_pages, pg->L, pg->page_size),
                     span(block_table, 4 * int64_t(pg->R) * pg->max_blocks),
                     span(q_start, 4 * (int64_t(pg->R) + 1)),
                     span(kv_lens, 4 * int64_t(pg->R)),
                     span(dev_status, 4)};
  for (const Span& x : in)
    if (overlap(o, x) || overlap(ws, x) || (lse != nullptr && overlap(s, x)))
      return fail(KVC_ERR_ALIAS, "out, lse and workspace may not overlap an input");
  if (overlap(o, ws) || (lse != nullptr && (overlap(s, o) || overlap(s, ws))))
    return fail(KVC_ERR_ALIAS, "out, lse and workspace may not overlap");
  AttnArgs a{};
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.q_tok = at->q_s_tok;
  a.q_head = at->q_s_head;
  a.o_tok = at->out_s_tok;
  a.o_head = at->out_s_head;
  a.pool[0] = to_view(pool_K);
  a.pool[1] = to_view(pool_V);
  a.table = block_table;
  a.q_start = q_start;
  a.kv_lens = kv_lens;
  a.R = pg->R;
  a.N = at->n_tokens;
  a.H = pg->H;
  a.G = at->n_q_heads / pg->H;
  a.d = pg->d;
  a.P = pg->n_pages;
  a.L = pg->L;
  a.B = pg->page_size;
  a.width = pg->max_blocks;
  a.layer = at->layer;
  a.causal = at->causal;
  // positions stay below 2^30: a window as long as that hides nothing, and the kernels'
  // sums of a position (down to -2^30) and a window stay within 32 bits
  a.window = at->window >= (1 << 30) ? 0 : at->window;
  a.scale_log2 = at->scale * 1.4426950408889634f;
  a.workspace = workspace;
  a.dev_status = dev_status;
  const cudaError_t e = pg->dtype == KVC_F32    ? launch_attn_f32(a, stream)
                        : attn_decode_fits(a) ? launch_attn_decode(a, stream)
                                              : launch_attn_tc(a, stream);
  if (e != cudaSuccess) return cuda_fail(e, "kvc_paged_attention launch");
  return KVC_OK;
}

}  // extern "C"
