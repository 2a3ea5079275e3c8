// C-ABI entry points of the paged attention operators (kda_paged.h): argument
// checks, launch plans, workspace carving.  Every check runs on the host before
// anything is queued.
#include <math.h>

#include <initializer_list>

#include "../../include/kda_paged.h"
#include "kda_paged.hpp"

#define KDA_API extern "C" __attribute__((visibility("default")))

namespace {

constexpr int64_t MAX_STRIDE = (int64_t)1 << 24;   // elements between tokens
constexpr int64_t MAX_KEYS = (int64_t)1 << 30;     // positions a table or a pool may hold
constexpr int64_t MAX_ROWS = (int64_t)1 << 25;     // (token, query head) rows of a call
constexpr int64_t MAX_TILES = (int64_t)1 << 24;    // row tiles of a call, over the kv heads
constexpr int MAX_SPLITS = 64;
constexpr size_t MAX_PARTIALS = (size_t)1 << 30;   // bytes of split partials

#define FAIL(status, ...) return (kda_status)kda::set_error(status, __VA_ARGS__)

bool misaligned(std::initializer_list<const void*> ps, size_t a) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & (a - 1)) return true;
  return false;
}

// Whether a buffer of `a` and one of `b` share bytes.
struct Span {
  const void* at;
  int64_t bytes;
};
bool overlap(std::initializer_list<Span> a, std::initializer_list<Span> b) {
  for (const Span& x : a)
    for (const Span& y : b) {
      const uintptr_t p = reinterpret_cast<uintptr_t>(x.at), q = reinterpret_cast<uintptr_t>(y.at);
      if (p != 0 && q != 0 && x.bytes > 0 && y.bytes > 0 && p < q + (uintptr_t)y.bytes &&
          q < p + (uintptr_t)x.bytes)
        return true;
    }
  return false;
}

size_t elem_size(int dtype) { return dtype == KDA_F32 ? 4 : 2; }

// What append and attention have in common: the pools.
kda_status check_pool(int dtype, int hkv, int dim, int page_size, int num_pages) {
  if (dtype != KDA_F32 && dtype != KDA_BF16 && dtype != KDA_F16)
    FAIL(KDA_ERR_DTYPE, "unknown dtype %d", dtype);
  if (hkv <= 0) FAIL(KDA_ERR_SHAPE, "head counts must be > 0");
  if (page_size < 1) FAIL(KDA_ERR_SHAPE, "page_size must be >= 1, got %d", page_size);
  if (num_pages <= 0) FAIL(KDA_ERR_SHAPE, "the cache must have at least one page");
  if (dim != 64 && dim != 128) FAIL(KDA_ERR_UNSUPPORTED, "head_dim must be 64 or 128, got %d", dim);
  if ((int64_t)num_pages * page_size > MAX_KEYS)
    FAIL(KDA_ERR_UNSUPPORTED, "num_pages * page_size above 2^30");
  if ((int64_t)hkv * dim > MAX_STRIDE) FAIL(KDA_ERR_UNSUPPORTED, "hkv * head_dim above 2^24");
  return KDA_OK;
}

// Resolves a token stride (0 = dense), in elements.
kda_status token_stride(const char* name, int64_t s, int64_t dense, size_t es, int64_t& out) {
  out = s ? s : dense;
  if (out < dense || out > MAX_STRIDE)
    FAIL(KDA_ERR_SHAPE, "%s %lld must be 0 or in [%lld, 2^24]", name, (long long)s, (long long)dense);
  if ((size_t)out * es % 16 != 0)
    FAIL(KDA_ERR_ARG, "%s %lld must keep rows 16-byte aligned", name, (long long)s);
  return KDA_OK;
}

// Resolves a page stride (0 = dense), to bytes.
kda_status page_stride(const char* name, int64_t s, int64_t dense, size_t es, int64_t& out) {
  if (s != 0 && (s < dense || s > (int64_t)1 << 40))
    FAIL(KDA_ERR_SHAPE, "%s %lld must be 0 or at least %lld", name, (long long)s, (long long)dense);
  out = (s ? s : dense) * (int64_t)es;
  if (out % 16 != 0) FAIL(KDA_ERR_ARG, "%s %lld must keep pages 16-byte aligned", name, (long long)s);
  return KDA_OK;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The workspace of split partials.
struct Plan {
  size_t o_bytes, lse_bytes, n_bytes;
};

kda_status check_attention(const kda_paged_attention_args* a, kda::AttnLaunch& L, Plan& p,
                           size_t& need) {
  if (!a) FAIL(KDA_ERR_ARG, "args is NULL");
  if (a->struct_size != sizeof(kda_paged_attention_args))
    FAIL(KDA_ERR_ARG, "struct_size %zu != sizeof(kda_paged_attention_args) %zu", a->struct_size,
         sizeof(kda_paged_attention_args));
  kda_status s = check_pool(a->dtype, a->hkv, a->head_dim, a->page_size, a->num_pages);
  if (s != KDA_OK) return s;
  if (a->n < 0) FAIL(KDA_ERR_SHAPE, "n must be >= 0");
  if (a->total_tokens < 0) FAIL(KDA_ERR_SHAPE, "total_tokens must be >= 0");
  if (a->hq <= 0) FAIL(KDA_ERR_SHAPE, "head counts must be > 0");
  if (a->hq % a->hkv != 0)
    FAIL(KDA_ERR_SHAPE, "hq (%d) must be divisible by hkv (%d)", a->hq, a->hkv);
  if (a->max_pages < 0) FAIL(KDA_ERR_SHAPE, "max_pages must be >= 0");
  if (a->table_stride != 0 && a->table_stride < a->max_pages)
    FAIL(KDA_ERR_SHAPE, "table_stride %lld must be 0 or at least max_pages", (long long)a->table_stride);
  if (a->window < 0 || a->sinks < 0) FAIL(KDA_ERR_SHAPE, "window and sinks must be >= 0");
  if (a->max_new_len < 0) FAIL(KDA_ERR_SHAPE, "max_new_len must be >= 0");
  if (a->splits < 0 || a->splits > MAX_SPLITS)
    FAIL(KDA_ERR_SHAPE, "splits must lie in [0, %d], got %d", MAX_SPLITS, a->splits);
  // hidden scores are -inf before the scale, which the kernels take times log2(e)
  if (!isfinite(a->scale * 1.4426950408889634f) || a->scale <= 0.0f)
    FAIL(KDA_ERR_SHAPE, "scale must be above 0 and finite in base two (below 2.35e38)");
  if ((int64_t)a->max_pages * a->page_size > MAX_KEYS)
    FAIL(KDA_ERR_UNSUPPORTED, "max_pages * page_size above 2^30");
  if ((int64_t)a->hq * a->head_dim > MAX_STRIDE)
    FAIL(KDA_ERR_UNSUPPORTED, "hq * head_dim above 2^24");
  // a launch holds fewer than 2^32 threads: 16 per row in the join, 256 per row tile
  if (a->total_tokens > MAX_ROWS / a->hq ||
      (a->total_tokens * (a->hq / a->hkv) / 16 + a->n) * a->hkv >= MAX_TILES)
    FAIL(KDA_ERR_UNSUPPORTED, "total_tokens * hq above 2^25, or row tiles above 2^24");
  const size_t es = elem_size(a->dtype);
  if ((s = token_stride("q_stride", a->q_stride, (int64_t)a->hq * a->head_dim, es, L.q_stride)) != KDA_OK)
    return s;
  const int64_t page = (int64_t)a->hkv * a->page_size * a->head_dim;
  if ((s = page_stride("k_page_stride", a->k_page_stride, page, es, L.k_page)) != KDA_OK) return s;
  if ((s = page_stride("v_page_stride", a->v_page_stride, page, es, L.v_page)) != KDA_OK) return s;
  L.table_stride = a->table_stride ? a->table_stride : a->max_pages;
  L.dtype = a->dtype; L.n = a->n; L.total = (int)a->total_tokens;
  L.hq = a->hq; L.hkv = a->hkv; L.group = a->hq / a->hkv; L.dim = a->head_dim;
  L.num_pages = a->num_pages; L.max_pages = a->max_pages;
  L.key_capacity = (int64_t)a->max_pages * a->page_size;
  L.page = kda::fast_div((uint32_t)a->page_size);
  L.gdiv = kda::fast_div((uint32_t)L.group);
  L.hdiv = kda::fast_div((uint32_t)L.hkv);
  // positions stay below 2^30, so larger windows and sink counts change nothing
  L.window = a->window < MAX_KEYS ? a->window : (int)MAX_KEYS;
  L.sinks = a->sinks < MAX_KEYS ? a->sinks : (int)MAX_KEYS;
  L.scale = a->scale;

  // Rows that a request may have, and keys that a row tile may visit.
  const int64_t most_new = a->max_new_len > 0 && a->max_new_len < a->total_tokens
                               ? a->max_new_len : a->total_tokens;
  int64_t keys = L.key_capacity;
  if (L.window > 0 && (int64_t)L.window + L.sinks + most_new < keys)
    keys = (int64_t)L.window + L.sinks + most_new;
  // The rows kernel serves calls whose requests have up to 32 rows per kv head, and short
  // fp32 ones; else all requests go through matrix tiles, the short ones beside the
  // chunks in one launch (33 mixed requests: 86 us against 101 us in a launch each, both
  // with a join 4 us slower than now).
  const int64_t most_rows = most_new * L.group, rows = a->total_tokens * a->hq;
  const int64_t group_rows = a->total_tokens * L.group;
  const bool tiles = a->dtype != KDA_F32 && most_rows > 32;
  L.row_blocks = most_rows > 16 ? 2 : 1;
  L.by_request = most_rows <= 32;
  // fp32 requests of 256 rows and more, on average, on 512 keys or more: workgroups of 128
  // rows (2048 tokens on 8192 keys, 8 heads on 2: 560 us against 690 us; 3 chunks of 840
  // tokens: 40.6 us against 44.2 us; but 8 requests of 128 rows on 2032 keys: 70 us against
  // 45 us, 40 of 33 rows: 420 us against 316 us, 200 tokens alone: 26.9 us against 19.6 us).
  L.chunks = a->dtype == KDA_F32 && !L.by_request && keys >= 512 &&
             group_rows >= (int64_t)a->n * 2 * kda::CHUNK_ROWS;
  // Eight waves (256 rows) a workgroup where key ranges are long and the rows fill the
  // chip with them, else four: kda_attn_tiles.hip says why, with both sides measured.
  L.tile_waves = !tiles ? 0 : keys >= 32768 && ceil_div(group_rows, 256) * a->hkv >= 256 ? 8 : 4;
  // Splits: pieces of long visits small enough to even out ragged lengths and to give
  // every compute unit work, in a grid that the many requests that are not split do not
  // swell.  A split row costs the tiles kernel its fp32 partials, so its rows are cut
  // only where they are few for the chip, ragged requests counting a third.
  int64_t units, grid;
  if (tiles) {
    units = ceil_div(group_rows, 32 * L.tile_waves) * a->hkv;
    // pieces of 2048 keys where requests are many (255 decodes beside a chunk of 512
    // tokens: 364 us, with 1024 keys 414 us), shorter ones where they are few (33 mixed
    // requests: 93 us with 1024 keys, 108 us with 2048; 512 tokens alone: 59 and 80 us)
    L.min_keys = units + (int64_t)a->n * a->hkv >= 2048 ? 2048 : units >= 256 ? 1024 : 512;
    grid = units >= (L.tile_waves == 8 ? 256 : 512) * (a->n > 1 ? 3 : 1) ? 0 : units >= 256 ? 8192 : 1024;
  } else {
    // chunks: 64 keys at least.  With 32, 64, 96, 128 and 256 keys 3 chunks of 840 tokens take
    // 51, 41, 48, 58 and 75 us, 300 tokens on 700 keys 27, 24, 31, 34 and 63 us, 4 fresh
    // ones of 512 tokens 67, 55, 53, 66 and 88 us; longer visits would like more: 8 of
    // 256 tokens on 1000 (64 channels) 77, 77, 70, 74 and 75 us, 2 of 400 tokens on 3000
    // 136, 133, 120, 106 and 92 us.
    units = L.by_request ? (int64_t)a->n * a->hkv
                         : ceil_div(group_rows, L.chunks ? kda::CHUNK_ROWS : 16 * L.row_blocks) * a->hkv;
    L.min_keys = units >= 1024 ? 2048 : units >= 256 ? 1024 : L.chunks ? 64 : 256;
    grid = L.by_request ? 16384 : 2048;
  }
  int64_t want = a->splits > 0 ? a->splits : units > 0 ? grid / units : 1;
  if (want > MAX_SPLITS) want = MAX_SPLITS;
  if (want > keys / L.min_keys) want = keys / L.min_keys;
  const int64_t cap = rows > 0 ? (int64_t)(MAX_PARTIALS / ((size_t)rows * a->head_dim * 4)) : 1;
  if (want > cap) want = cap;
  L.splits = want > 1 ? (int)want : 1;
  p.o_bytes = p.lse_bytes = p.n_bytes = 0;
  if (L.splits > 1) {
    p.o_bytes = (size_t)L.splits * rows * a->head_dim * 4;
    p.lse_bytes = ((size_t)L.splits * rows * 4 + 15) / 16 * 16;
    p.n_bytes = ((size_t)rows * 4 + 15) / 16 * 16;
  }
  // at most 2^30 of partials, a 64th of it of log-sum-exps and, two splits or more, half
  // of that of counts: KDA_PAGED_ATTENTION_WORKSPACE_MAX
  need = p.o_bytes + p.lse_bytes + p.n_bytes;
  return KDA_OK;
}

}  // namespace

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

KDA_API kda_status kda_paged_attention_workspace_size(const kda_paged_attention_args* a, size_t* bytes) {
  if (!bytes) FAIL(KDA_ERR_ARG, "bytes is NULL");
  kda::AttnLaunch L = {};
  Plan p;
  const kda_status s = check_attention(a, L, p, *bytes);
  return s == KDA_OK ? (kda_status)kda::set_ok() : s;
}

KDA_API kda_status kda_paged_attention(const kda_paged_attention_args* a) {
  kda::AttnLaunch L = {};
  Plan p;
  size_t need = 0;
  const kda_status s = check_attention(a, L, p, need);
  if (s != KDA_OK) return s;
  if (misaligned({a->q, a->k_cache, a->v_cache, a->out, a->workspace}, 16))
    FAIL(KDA_ERR_ARG, "tensor base pointers must be 16-byte aligned");
  if (misaligned({a->block_table, a->cu_seqlens, a->seq_lens, a->lse}, 4))
    FAIL(KDA_ERR_ARG, "index arrays and lse must be 4-byte aligned");
  if (a->n == 0 || a->total_tokens == 0) return (kda_status)kda::set_ok();
  if (!a->q || !a->k_cache || !a->v_cache || !a->cu_seqlens || !a->seq_lens || !a->out ||
      (!a->block_table && a->max_pages > 0))
    FAIL(KDA_ERR_ARG,
         "q, k_cache, v_cache, block_table, cu_seqlens, seq_lens and out must be non-NULL");
  if (need > 0 && (a->workspace == nullptr || a->workspace_bytes < need))
    FAIL(KDA_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need,
         a->workspace ? a->workspace_bytes : (size_t)0);
  L.q = a->q; L.kc = a->k_cache; L.vc = a->v_cache;
  L.table = a->block_table; L.cu = a->cu_seqlens; L.seq = a->seq_lens;
  L.out = a->out; L.lse = a->lse;
  if (need > 0) {
    char* ws = (char*)a->workspace;
    L.part_o = (float*)ws;
    L.part_lse = (float*)(ws + p.o_bytes);
    L.part_n = (int32_t*)(ws + p.o_bytes + p.lse_bytes);
  }
  L.stream = a->stream;
  hipError_t e = L.tile_waves > 0 ? kda::launch_attn_tiles(L)
                 : L.chunks       ? kda::launch_attn_chunks(L)
                                  : kda::launch_attn_rows(L);
  if (e == hipSuccess && need > 0) e = kda::launch_attn_join(L);
  if (e != hipSuccess) FAIL(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  return (kda_status)kda::set_ok();
}
