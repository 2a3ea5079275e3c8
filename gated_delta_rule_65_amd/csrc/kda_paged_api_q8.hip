// C-ABI entry points of the paged cache in 8 bits (kda_paged_q8.h): argument checks and
// launch plans.  Every check runs on the host before anything is queued.
#include "../../include/kda_paged_q8.h"
#include "kda_attn_q8.hpp"
#include "kda_paged_api.hpp"

namespace {

// Workgroups of a call that moves rows: up to 256 threads each, and a launch holds fewer than 2^32.
constexpr int64_t MAX_UNITS = ((int64_t)1 << 24) - 1;

kda_status check_codes(int code, int page_size, int block) {
  if (code != KDA_E4M3 && code != KDA_INT8) FAIL(KDA_ERR_DTYPE, "unknown code %d", code);
  if (block < 1 || page_size % block != 0)
    FAIL(KDA_ERR_SHAPE, "block must be a divisor of page_size (%d), got %d", page_size, block);
  return KDA_OK;
}

// What append and read have in common.
template <typename A> kda_status check_rows(const A* a, kda::CacheQ8Launch& L) {
  kda_status s = check_pool(a->dtype, a->hkv, a->head_dim, a->page_size, a->num_pages);
  if (s != KDA_OK || (s = check_codes(a->code, a->page_size, a->block)) != KDA_OK) return s;
  if (a->n < 0) FAIL(KDA_ERR_SHAPE, "n must be >= 0");
  if (a->total_tokens < 0) FAIL(KDA_ERR_SHAPE, "total_tokens must be >= 0");
  if (a->max_pages < 0) FAIL(KDA_ERR_SHAPE, "max_pages must be >= 0");
  if (a->table_stride != 0 && a->table_stride < a->max_pages)
    FAIL(KDA_ERR_SHAPE, "table_stride %lld must be 0 or at least max_pages", (long long)a->table_stride);
  if ((int64_t)a->max_pages * a->page_size > MAX_KEYS)
    FAIL(KDA_ERR_UNSUPPORTED, "max_pages * page_size above 2^30");
  if (a->total_tokens > INT32_MAX) FAIL(KDA_ERR_UNSUPPORTED, "total_tokens above 2^31-1");
  const int64_t page = (int64_t)a->hkv * a->page_size * a->head_dim;
  if ((s = page_stride("k_page_stride", a->k_page_stride, page, 1, L.k_page)) != KDA_OK) return s;
  if ((s = page_stride("v_page_stride", a->v_page_stride, page, 1, L.v_page)) != KDA_OK) return s;
  if (misaligned({a->k_cache, a->v_cache}, 16))
    FAIL(KDA_ERR_ARG, "tensor base pointers must be 16-byte aligned");
  if (misaligned({a->k_scale, a->v_scale, a->block_table, a->cu_seqlens, a->seq_lens}, 4))
    FAIL(KDA_ERR_ARG, "scales and index arrays must be 4-byte aligned");
  L.kc = (void*)a->k_cache; L.vc = (void*)a->v_cache;
  L.ks = (float*)a->k_scale; L.vs = (float*)a->v_scale;
  L.table = a->block_table; L.cu = a->cu_seqlens; L.seq = a->seq_lens;
  L.table_stride = a->table_stride ? a->table_stride : a->max_pages;
  L.capacity = (int64_t)a->max_pages * a->page_size;
  L.dtype = a->dtype; L.code = a->code; L.n = a->n; L.total = (int)a->total_tokens;
  L.hkv = a->hkv; L.dim = a->head_dim; L.num_pages = a->num_pages; L.max_pages = a->max_pages;
  L.per_page = a->page_size / a->block;
  L.page = kda::fast_div((uint32_t)a->page_size);
  L.block = kda::fast_div((uint32_t)a->block);
  L.hdiv = kda::fast_div((uint32_t)a->hkv);
  L.stream = a->stream;
  return KDA_OK;
}
template <typename A> kda_status check_present(const A* a) {
  if (!a->k_cache || !a->v_cache || !a->k_scale || !a->v_scale || !a->cu_seqlens || !a->seq_lens ||
      (!a->block_table && a->max_pages > 0))
    FAIL(KDA_ERR_ARG,
         "k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens and seq_lens must be non-NULL");
  return KDA_OK;
}

// The arguments as those of an attention over a cache of q's type.
kda_paged_attention_args plain(const kda_paged_attention_q8_args* a) {
  kda_paged_attention_args b = {};
  b.struct_size = sizeof(b);
  b.q = a->q; b.k_cache = a->k_cache; b.v_cache = a->v_cache;
  b.block_table = a->block_table; b.cu_seqlens = a->cu_seqlens; b.seq_lens = a->seq_lens;
  b.out = a->out; b.lse = a->lse;
  b.workspace = a->workspace; b.workspace_bytes = a->workspace_bytes;
  b.total_tokens = a->total_tokens; b.q_stride = a->q_stride;
  b.k_page_stride = a->k_page_stride; b.v_page_stride = a->v_page_stride;
  b.table_stride = a->table_stride;
  b.dtype = a->dtype; b.n = a->n; b.hq = a->hq; b.hkv = a->hkv;
  b.head_dim = a->head_dim; b.page_size = a->page_size; b.num_pages = a->num_pages;
  b.max_pages = a->max_pages; b.window = a->window; b.sinks = a->sinks;
  b.max_new_len = a->max_new_len; b.splits = a->splits; b.scale = a->scale; b.stream = a->stream;
  return b;
}

kda_status check_q8(const kda_paged_attention_q8_args* a, kda_paged_attention_args& b,
                    kda::AttnQ8Launch& L, Plan& p, size_t& need) {
  if (!a) FAIL(KDA_ERR_ARG, "args is NULL");
  if (a->struct_size != sizeof(kda_paged_attention_q8_args))
    FAIL(KDA_ERR_ARG, "struct_size %zu != sizeof(kda_paged_attention_q8_args) %zu", a->struct_size,
         sizeof(kda_paged_attention_q8_args));
  if (a->dtype == KDA_F32)
    FAIL(KDA_ERR_DTYPE, "attention over a cache in 8 bits takes bf16 or fp16 rows");
  b = plain(a);
  kda_status s = check_attention(&b, L, p, need, 1);
  if (s != KDA_OK || (s = check_codes(a->code, a->page_size, a->block)) != KDA_OK) return s;
  L.code = a->code;
  L.scales.k = a->k_scale; L.scales.v = a->v_scale;
  L.scales.block = kda::fast_div((uint32_t)a->block);
  L.scales.per_page = a->page_size / a->block;
  return KDA_OK;
}

}  // namespace

KDA_API kda_status kda_kv_append_q8(const kda_kv_append_q8_args* a) {
  if (!a) FAIL(KDA_ERR_ARG, "args is NULL");
  if (a->struct_size != sizeof(kda_kv_append_q8_args))
    FAIL(KDA_ERR_ARG, "struct_size %zu != sizeof(kda_kv_append_q8_args) %zu", a->struct_size,
         sizeof(kda_kv_append_q8_args));
  kda::CacheQ8Launch L = {};
  kda_status s = check_rows(a, L);
  if (s != KDA_OK) return s;
  if ((a->total_tokens / a->block + 2 * (int64_t)a->n) * a->hkv > MAX_UNITS)
    FAIL(KDA_ERR_UNSUPPORTED, "blocks of rows, over the heads, not below 2^24");
  const size_t es = elem_size(a->dtype);
  const int64_t dense = (int64_t)a->hkv * a->head_dim;
  int64_t ks, vs;
  if ((s = token_stride("k_stride", a->k_stride, dense, es, ks)) != KDA_OK) return s;
  if ((s = token_stride("v_stride", a->v_stride, dense, es, vs)) != KDA_OK) return s;
  if (misaligned({a->k, a->v}, 16)) FAIL(KDA_ERR_ARG, "tensor base pointers must be 16-byte aligned");
  if (a->n == 0 || a->total_tokens == 0) return (kda_status)kda::set_ok();
  if (!a->k || !a->v) FAIL(KDA_ERR_ARG, "k and v must be non-NULL");
  if ((s = check_present(a)) != KDA_OK) return s;
  L.k = a->k; L.v = a->v;
  L.k_stride = ks * (int64_t)es; L.v_stride = vs * (int64_t)es;
  const hipError_t e = kda::launch_append_q8(L);
  if (e != hipSuccess) FAIL(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  return (kda_status)kda::set_ok();
}

KDA_API kda_status kda_kv_read_q8(const kda_kv_read_q8_args* a) {
  if (!a) FAIL(KDA_ERR_ARG, "args is NULL");
  if (a->struct_size != sizeof(kda_kv_read_q8_args))
    FAIL(KDA_ERR_ARG, "struct_size %zu != sizeof(kda_kv_read_q8_args) %zu", a->struct_size,
         sizeof(kda_kv_read_q8_args));
  kda::CacheQ8Launch L = {};
  kda_status s = check_rows(a, L);
  if (s != KDA_OK) return s;
  if (a->total_tokens / 4 + a->n > MAX_UNITS)
    FAIL(KDA_ERR_UNSUPPORTED, "total_tokens near 2^26, or requests near 2^24");
  if (misaligned({a->k_out, a->v_out}, 16))
    FAIL(KDA_ERR_ARG, "tensor base pointers must be 16-byte aligned");
  if (a->n == 0 || a->total_tokens == 0) return (kda_status)kda::set_ok();
  if (!a->k_out || !a->v_out) FAIL(KDA_ERR_ARG, "k_out and v_out must be non-NULL");
  if ((s = check_present(a)) != KDA_OK) return s;
  L.ko = a->k_out; L.vo = a->v_out;
  const hipError_t e = kda::launch_read_q8(L);
  if (e != hipSuccess) FAIL(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  return (kda_status)kda::set_ok();
}

KDA_API kda_status kda_paged_attention_q8_workspace_size(const kda_paged_attention_q8_args* a,
                                                         size_t* bytes) {
  if (!bytes) FAIL(KDA_ERR_ARG, "bytes is NULL");
  kda_paged_attention_args b;
  kda::AttnQ8Launch L = {};
  Plan p;
  const kda_status s = check_q8(a, b, L, p, *bytes);
  return s == KDA_OK ? (kda_status)kda::set_ok() : s;
}

KDA_API kda_status kda_paged_attention_q8(const kda_paged_attention_q8_args* a) {
  kda_paged_attention_args b;
  kda::AttnQ8Launch L = {};
  Plan p;
  size_t need = 0;
  bool go = false;
  kda_status s = check_q8(a, b, L, p, need);
  if (s != KDA_OK) return s;
  if (misaligned({a->k_scale, a->v_scale}, 4)) FAIL(KDA_ERR_ARG, "scales must be 4-byte aligned");
  if ((s = check_call(&b, L, p, need, go)) != KDA_OK) return s;
  if (!go) return (kda_status)kda::set_ok();
  if (!a->k_scale || !a->v_scale) FAIL(KDA_ERR_ARG, "k_scale and v_scale must be non-NULL");
  hipError_t e = L.tile_waves > 0 ? kda::launch_attn_q8_tiles(L) : kda::launch_attn_q8_rows(L);
  if (e == hipSuccess && need > 0) e = kda::launch_attn_join(L);
  if (e != hipSuccess) FAIL(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  return (kda_status)kda::set_ok();
}
