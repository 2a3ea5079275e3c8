// Block tables and slot maps of a step from the request lengths, and the new
// key and value rows into their cache slots.
//
// Tables.  One launch: each workgroup owns 1024 consecutive new tokens and walks the
// requests 1024 at a time, with a prefix sum of (new tokens, missing pages) in LDS,
// until it has placed all of its own.  Every workgroup repeats the walk, which takes a
// scan per 1024 requests, and so needs no second launch.  A new page is entered by
// the token that opens it, or by the first workgroup where that token lies past the
// slot map's room, and its id comes from the free list, never from the table, so
// workgroups do not depend on one another.  Bound by latency: 256 requests of one
// token 3.9 us, 1000 requests with 93766 tokens 5.6 us.
//
// Append.  A copy of 16-byte pieces, bound by HBM: 32768 tokens of 8 heads of 128 fp16
// channels (134 MB read, 134 MB written) 53 us, 5.0 TB/s; a large copy reaches 4.8.  (42 us
// where the last-level cache still holds the same rows from the call before.)
#include "kda_common.hpp"
#include "kda_paged.hpp"

namespace kda {
namespace {

constexpr int NT = 1024;

__device__ __forceinline__ uint32_t pdiv(uint32_t t, const FastDiv& f) {
  return __umulhi(2u * t, f.mul) >> f.shift;
}
// Pages of t tokens.
__device__ __forceinline__ int pages_of(uint32_t t, const FastDiv& f) {
  t &= 0x7fffffffu;
  const uint32_t p = pdiv(t, f);
  return (int)(p + (p * f.d < t));
}

__global__ __launch_bounds__(NT) void page_tables_kernel(const TablesLaunch a) {
  __shared__ int s_cu[NT + 1], s_ctx[NT], s_have[NT], s_first[NT];
  __shared__ int w_tok[NT / 64], w_page[NT / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * NT;
  const int64_t t = t0 + tid;
  const bool room = t < a.max_tokens;
  bool placed = false;
  int64_t tok_base = 0, page_base = 0;
  for (int r0 = 0; r0 < a.n; r0 += NT) {
    const int i = r0 + tid;
    int ctx = 0, fresh = 0;
    if (i < a.n) {
      ctx = max(a.context[i], 0);
      fresh = max(a.fresh[i], 0);
    }
    const int have = pages_of((uint32_t)ctx, a.page);
    const uint32_t total = (uint32_t)ctx + (uint32_t)fresh;
    const int need = pages_of(total, a.page) - have;
    // inclusive sums over the wave, then over the waves
    int x = fresh, y = need;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(x, d), v = __shfl_up(y, d);
      if (lane >= d) {
        x += u;
        y += v;
      }
    }
    if (lane == 63) {
      w_tok[wave] = x;
      w_page[wave] = y;
    }
    __syncthreads();
    int bx = 0, by = 0, sx = 0, sy = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
      const int u = w_tok[w], v = w_page[w];
      if (w < wave) {
        bx += u;
        by += v;
      }
      sx += u;
      sy += v;
    }
    s_cu[tid] = bx + x - fresh;
    if (tid == 0) s_cu[NT] = sx;
    s_ctx[tid] = ctx;
    s_have[tid] = have;
    s_first[tid] = (int)(page_base + by + y - need);
    if (blockIdx.x == 0 && i < a.n) {
      a.cu[i] = (int32_t)(tok_base + bx + x - fresh);
      a.seq[i] = (int32_t)total;
    }
    __syncthreads();
    if (room && !placed && t - tok_base < s_cu[NT]) {
      placed = true;
      const int u = (int)(t - tok_base);
      // the last request of this block that starts at or before token u
      int lo = 0, hi = min(NT, a.n - r0);
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= u) lo = mid;
        else hi = mid;
      }
      const int pos = s_ctx[lo] + (u - s_cu[lo]);
      const int page = (int)pdiv((uint32_t)pos & 0x7fffffffu, a.page);
      const int off = pos - page * (int)a.page.d;
      int id = -1;
      if (pos >= 0 && page < a.max_pages) {
        int32_t* entry = a.table + (int64_t)(r0 + lo) * a.table_stride + page;
        if (page >= s_have[lo]) {
          const int64_t f = (int64_t)s_first[lo] + (page - s_have[lo]);
          if (f >= 0 && f < a.num_free) id = a.free_pages[f];
          if (off == 0) *entry = id;
        } else {
          id = *entry;
        }
      }
      a.slots[t] = (uint32_t)id < (uint32_t)a.num_pages ? (int64_t)id * a.page.d + off : -1;
      if (a.positions != nullptr) a.positions[t] = pos;
    }
    if (__builtin_expect(blockIdx.x == 0 && tok_base + sx > a.max_tokens, 0)) {
      // the pages [late, end) of the lane's request open past the room, where no thread has
      // their token: the wave goes through its requests with such pages, 64 pages at a time
      const int64_t left = a.max_tokens - (tok_base + bx + x - fresh);  // room for its tokens
      const int late = pages_of((uint32_t)ctx + (uint32_t)min((int64_t)fresh, max(left, (int64_t)0)), a.page);
      const int end = min(have + need, a.max_pages);
      for (uint64_t some = __ballot(late < end); some != 0; some &= some - 1) {
        const int l = __builtin_ctzll(some);
        const int last = __shfl(end, l), held = __shfl(have, l);
        const int64_t first = __shfl((int)(page_base + by + y - need), l);
        int32_t* row = a.table + (int64_t)(i - lane + l) * a.table_stride;
        for (int p = __shfl(late, l) + lane; p < last; p += 64) {
          const int64_t f = first + (p - held);
          row[p] = f >= 0 && f < a.num_free ? a.free_pages[f] : -1;
        }
      }
    }
    tok_base += s_cu[NT];
    page_base += sy;
    __syncthreads();
    // nothing further on concerns a workgroup whose tokens are all placed (the
    // first one goes on: it writes the offsets and the totals)
    if (blockIdx.x != 0 && tok_base >= t0 + NT) return;
  }
  if (room && !placed) {
    a.slots[t] = -1;
    if (a.positions != nullptr) a.positions[t] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.cu[a.n] = (int32_t)tok_base;
    a.taken[0] = (int32_t)page_base;
  }
}

__global__ __launch_bounds__(256) void kv_append_kernel(const AppendLaunch a, FastDiv per_token,
                                                        FastDiv per_row) {
  const uint32_t x = blockIdx.x * 256u + threadIdx.x;
  if (x >= a.tokens * per_token.d) return;
  const uint32_t t = pdiv(x, per_token);
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= a.num_slots) return;
  const uint32_t p = x - t * per_token.d;  // piece of the token's row of all heads
  const uint32_t h = pdiv(p, per_row), c = p - h * per_row.d;
  const uint32_t page = pdiv((uint32_t)slot, a.page), off = (uint32_t)slot - page * a.page.d;
  const int64_t in = 16 * (int64_t)p, head = ((int64_t)h * a.page.d + off) * a.row_bytes + 16 * (int64_t)c;
  const uint4 k = *reinterpret_cast<const uint4*>((const char*)a.k + t * a.k_stride + in);
  const uint4 v = *reinterpret_cast<const uint4*>((const char*)a.v + t * a.v_stride + in);
  *reinterpret_cast<uint4*>((char*)a.kc + page * a.k_page + head) = k;
  *reinterpret_cast<uint4*>((char*)a.vc + page * a.v_page + head) = v;
}

}  // namespace

hipError_t launch_page_tables(const TablesLaunch& L) {
  const unsigned blocks = (unsigned)((L.max_tokens + NT - 1) / NT);
  hipLaunchKernelGGL(page_tables_kernel, dim3(blocks ? blocks : 1), dim3(NT), 0,
                     (hipStream_t)L.stream, L);
  return hipGetLastError();
}

hipError_t launch_kv_append(const AppendLaunch& L) {
  const uint32_t per_row = (uint32_t)L.row_bytes / 16, per_token = per_row * (uint32_t)L.hkv;
  const int64_t pieces = L.tokens * per_token;
  hipLaunchKernelGGL(kv_append_kernel, dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0,
                     (hipStream_t)L.stream, L, fast_div(per_token), fast_div(per_row));
  return hipGetLastError();
}

}  // namespace kda
