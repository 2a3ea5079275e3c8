// Host-side launch descriptors of the paged attention entry points.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

// t / d for 0 <= t < 2^31 as mulhi(2 t, mul) >> shift: with shift = ceil(log2 d)
// and mul = ceil(2^(31 + shift) / d), the error mul * d - 2^(31 + shift) is below
// 2^shift, which t < 2^31 keeps out of the quotient.
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f;
  f.d = d;
  f.shift = 0;
  while (((uint64_t)1 << f.shift) < d) ++f.shift;
  f.mul = (uint32_t)((((uint64_t)1 << (31 + f.shift)) + d - 1) / d);
  return f;
}

// Block tables and slot maps of a step.
struct TablesLaunch {
  const int32_t *context, *fresh;  // [n] cached and new tokens per request
  const int32_t* free_pages;       // [num_free]
  int32_t* table;                  // [n, max_pages], row stride table_stride
  int64_t table_stride;
  int64_t* slots;                  // [max_tokens]
  int32_t* positions;              // [max_tokens] or NULL
  int32_t *cu, *seq, *taken;       // [n + 1], [n], [1]
  int64_t max_tokens;
  int n, num_free, max_pages, num_pages;
  FastDiv page;
  void* stream;
};
hipError_t launch_page_tables(const TablesLaunch& L);

// New K and V rows into their cache slots.
struct AppendLaunch {
  const void *k, *v;
  void *kc, *vc;
  const int64_t* slots;        // [tokens]
  int64_t tokens;
  int64_t k_stride, v_stride;  // bytes between tokens
  int64_t k_page, v_page;      // bytes between pages
  int hkv, row_bytes;          // bytes of one head's row
  int64_t num_slots;           // num_pages * page size
  FastDiv page;
  void* stream;
};
hipError_t launch_kv_append(const AppendLaunch& L);

// Attention over the paged cache.
struct AttnLaunch {
  const void *q, *kc, *vc;
  const int32_t *table, *cu, *seq;
  void* out;
  float* lse;              // [T, hq] or NULL
  // split partials (splits > 1), token-major: part_o [splits][T * hq][dim] fp32
  // normalised outputs, part_lse [splits][T * hq] base-2 log-sum-exp, part_n [T * hq]
  // the splits that each row was cut into
  float *part_o, *part_lse;
  int32_t* part_n;
  int64_t q_stride;        // elements between tokens
  int64_t k_page, v_page;  // bytes between pages
  int64_t table_stride;
  int dtype, n, total, hq, hkv, group, dim, num_pages, max_pages;
  int64_t key_capacity;    // max_pages * page size
  FastDiv page, gdiv, hdiv;  // by the page size, the group, hkv
  int window, sinks;       // window 0: every earlier key
  float scale;
  int tile_waves;          // tiles kernel: waves of 32 rows (4 or 8); 0: another one runs
  int row_blocks;          // rows kernel: 16-row blocks per wave (1 or 2)
  int by_request;          // rows kernel: a workgroup per request, not per row tile
  int chunks;              // the fp32 chunks kernel runs, not the rows kernel
  int splits, min_keys;    // splits of a visit at most, and keys of one at least
  void* stream;
};
constexpr int CHUNK_ROWS = 128;  // rows of a workgroup of the fp32 chunks
hipError_t launch_attn_rows(const AttnLaunch& L);
hipError_t launch_attn_tiles(const AttnLaunch& L);
hipError_t launch_attn_chunks(const AttnLaunch& L);
hipError_t launch_attn_join(const AttnLaunch& L);

// Stores the calling thread's error text (kda_last_error) and returns status.
int set_error(int status, const char* fmt, ...);
int set_ok();

}  // namespace kda
