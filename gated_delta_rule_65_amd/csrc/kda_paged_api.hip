// C-ABI entry points of the paged attention operators (kda_paged.h): argument
// checks, launch plans, workspace carving.  Every check runs on the host before
// anything is queued.
#include "kda_paged_api.hpp"

KDA_API kda_status kda_page_tables(const kda_page_tables_args* a) {
  if (!a) FAIL(KDA_ERR_ARG, "args is NULL");
  if (a->struct_size != sizeof(kda_page_tables_args))
    FAIL(KDA_ERR_ARG, "struct_size %zu != sizeof(kda_page_tables_args) %zu", a->struct_size,
         sizeof(kda_page_tables_args));
  if (a->n < 0) FAIL(KDA_ERR_SHAPE, "n must be >= 0");
  if (a->num_free < 0) FAIL(KDA_ERR_SHAPE, "num_free must be >= 0");
  if (a->max_pages < 0) FAIL(KDA_ERR_SHAPE, "max_pages must be >= 0");
  if (a->num_pages < 0) FAIL(KDA_ERR_SHAPE, "num_pages must be >= 0");
  if (a->page_size < 1) FAIL(KDA_ERR_SHAPE, "page_size must be >= 1, got %d", a->page_size);
  if (a->max_tokens < 0) FAIL(KDA_ERR_SHAPE, "max_tokens must be >= 0");
  if (a->table_stride != 0 && a->table_stride < a->max_pages)
    FAIL(KDA_ERR_SHAPE, "table_stride %lld must be 0 or at least max_pages", (long long)a->table_stride);
  if ((int64_t)a->num_pages * a->page_size > MAX_KEYS ||
      (int64_t)a->max_pages * a->page_size > MAX_KEYS || a->max_tokens > MAX_KEYS)
    FAIL(KDA_ERR_UNSUPPORTED,
         "num_pages * page_size, max_pages * page_size and max_tokens must stay within 2^30");
  if (!a->cu_seqlens || !a->pages_taken)
    FAIL(KDA_ERR_ARG, "cu_seqlens and pages_taken must be non-NULL");
  if (a->n > 0 && (!a->context_lens || !a->new_lens || !a->seq_lens))
    FAIL(KDA_ERR_ARG, "context_lens, new_lens and seq_lens must be non-NULL");
  if (a->n > 0 && a->max_pages > 0 && !a->block_table) FAIL(KDA_ERR_ARG, "block_table must be non-NULL");
  if (a->num_free > 0 && !a->free_pages) FAIL(KDA_ERR_ARG, "free_pages must be non-NULL");
  if (a->max_tokens > 0 && !a->slot_mapping) FAIL(KDA_ERR_ARG, "slot_mapping must be non-NULL");
  if (misaligned({a->context_lens, a->new_lens, a->free_pages, a->block_table, a->positions,
                  a->cu_seqlens, a->seq_lens, a->pages_taken}, 4) ||
      misaligned({a->slot_mapping}, 8))
    FAIL(KDA_ERR_ARG, "index arrays must be aligned to their elements");
  // the first workgroup writes lengths that the others may have yet to read
  const int64_t n4 = 4 * (int64_t)a->n, stride = a->table_stride ? a->table_stride : a->max_pages;
  const Span table = {a->block_table, a->n > 0 ? 4 * ((a->n - 1) * stride + a->max_pages) : 0};
  const Span lens[] = {{a->context_lens, n4}, {a->new_lens, n4}, {a->free_pages, 4 * (int64_t)a->num_free}};
  if (overlap({lens[0], lens[1], lens[2], table},
              {{a->cu_seqlens, n4 + 4}, {a->seq_lens, n4}, {a->pages_taken, 4},
               {a->slot_mapping, 8 * a->max_tokens}, {a->positions, 4 * a->max_tokens}}) ||
      overlap({lens[0], lens[1], lens[2]}, {table}))
    FAIL(KDA_ERR_ARG, "outputs must not overlap inputs (a step's seq_lens are not its context_lens)");
  kda::TablesLaunch L;
  L.context = a->context_lens; L.fresh = a->new_lens; L.free_pages = a->free_pages;
  L.table = a->block_table;
  L.table_stride = stride;
  L.slots = a->slot_mapping; L.positions = a->positions;
  L.cu = a->cu_seqlens; L.seq = a->seq_lens; L.taken = a->pages_taken;
  L.max_tokens = a->max_tokens;
  L.n = a->n; L.num_free = a->num_free; L.max_pages = a->max_pages; L.num_pages = a->num_pages;
  L.page = kda::fast_div((uint32_t)a->page_size);
  L.stream = a->stream;
  const hipError_t e = kda::launch_page_tables(L);
  if (e != hipSuccess) FAIL(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  return (kda_status)kda::set_ok();
}

KDA_API kda_status kda_kv_append(const kda_kv_append_args* a) {
  if (!a) FAIL(KDA_ERR_ARG, "args is NULL");
  if (a->struct_size != sizeof(kda_kv_append_args))
    FAIL(KDA_ERR_ARG, "struct_size %zu != sizeof(kda_kv_append_args) %zu", a->struct_size,
         sizeof(kda_kv_append_args));
  kda_status s = check_pool(a->dtype, a->hkv, a->head_dim, a->page_size, a->num_pages);
  if (s != KDA_OK) return s;
  if (a->total_tokens < 0) FAIL(KDA_ERR_SHAPE, "total_tokens must be >= 0");
  const size_t es = elem_size(a->dtype);
  const int64_t dense = (int64_t)a->hkv * a->head_dim;
  if (a->total_tokens > (int64_t)INT32_MAX / (dense * (int64_t)es / 16))
    FAIL(KDA_ERR_UNSUPPORTED, "total_tokens * hkv * head_dim above 2^31-1 16-byte pieces");
  int64_t ks, vs, kp, vp;
  if ((s = token_stride("k_stride", a->k_stride, dense, es, ks)) != KDA_OK) return s;
  if ((s = token_stride("v_stride", a->v_stride, dense, es, vs)) != KDA_OK) return s;
  if ((s = page_stride("k_page_stride", a->k_page_stride, dense * a->page_size, es, kp)) != KDA_OK) return s;
  if ((s = page_stride("v_page_stride", a->v_page_stride, dense * a->page_size, es, vp)) != KDA_OK) return s;
  if (misaligned({a->k, a->v, a->k_cache, a->v_cache}, 16))
    FAIL(KDA_ERR_ARG, "tensor base pointers must be 16-byte aligned");
  if (misaligned({a->slot_mapping}, 8)) FAIL(KDA_ERR_ARG, "slot_mapping must be 8-byte aligned");
  if (a->total_tokens == 0) return (kda_status)kda::set_ok();
  if (!a->k || !a->v || !a->k_cache || !a->v_cache || !a->slot_mapping)
    FAIL(KDA_ERR_ARG, "k, v, k_cache, v_cache and slot_mapping must be non-NULL");
  kda::AppendLaunch L;
  L.k = a->k; L.v = a->v; L.kc = a->k_cache; L.vc = a->v_cache;
  L.slots = a->slot_mapping; L.tokens = a->total_tokens;
  L.k_stride = ks * (int64_t)es; L.v_stride = vs * (int64_t)es;
  L.k_page = kp; L.v_page = vp;
  L.hkv = a->hkv; L.row_bytes = a->head_dim * (int)es;
  L.num_slots = (int64_t)a->num_pages * a->page_size;
  L.page = kda::fast_div((uint32_t)a->page_size);
  L.stream = a->stream;
  const hipError_t e = kda::launch_kv_append(L);
  if (e != hipSuccess) FAIL(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  return (kda_status)kda::set_ok();
}

// The struct and what the call's plan follows from it.
static kda_status check(const kda_paged_attention_args* a, kda::AttnLaunch& L, Plan& p, size_t& need) {
  if (!a) FAIL(KDA_ERR_ARG, "args is NULL");
  if (a->struct_size != sizeof(kda_paged_attention_args))
    FAIL(KDA_ERR_ARG, "struct_size %zu != sizeof(kda_paged_attention_args) %zu", a->struct_size,
         sizeof(kda_paged_attention_args));
  return check_attention(a, L, p, need);
}

KDA_API kda_status kda_paged_attention_workspace_size(const kda_paged_attention_args* a, size_t* bytes) {
  if (!bytes) FAIL(KDA_ERR_ARG, "bytes is NULL");
  kda::AttnLaunch L = {};
  Plan p;
  const kda_status s = check(a, L, p, *bytes);
  return s == KDA_OK ? (kda_status)kda::set_ok() : s;
}

KDA_API kda_status kda_paged_attention(const kda_paged_attention_args* a) {
  kda::AttnLaunch L = {};
  Plan p;
  size_t need = 0;
  bool go = false;
  kda_status s = check(a, L, p, need);
  if (s != KDA_OK || (s = check_call(a, L, p, need, go)) != KDA_OK) return s;
  if (!go) return (kda_status)kda::set_ok();
  hipError_t e = L.tile_waves > 0 ? kda::launch_attn_tiles(L)
                 : L.chunks       ? kda::launch_attn_chunks(L)
                                  : kda::launch_attn_rows(L);
  if (e == hipSuccess && need > 0) e = kda::launch_attn_join(L);
  if (e != hipSuccess) FAIL(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  return (kda_status)kda::set_ok();
}
