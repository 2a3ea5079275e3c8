// Device helpers shared by the paged attention kernels (gfx950, wave64).
//
// A request's rows are its (new token, query head of the group) pairs of one
// kv head: row r is token r / G, head r % G, so that a tile of rows reads each
// key once for the whole group.  The scores are formed transposed, S^T = K Q^T:
// a lane then holds several keys of one row (the MFMA column), its softmax
// statistics need no more than a swap between lane groups, and the C layout of
// S^T is, up to a permutation of the keys, the B layout of P^T in
// O^T = V^T P^T.  V^T comes out of the row-major V tile in LDS with the
// transposing 8-byte read.
#pragma once
#include "kda_mfma.hpp"
#include "kda_paged.hpp"

namespace kda {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4v_t __attribute__((ext_vector_type(4)));

constexpr float NEG_INF = -__builtin_inff();
constexpr float LN2 = 0.6931471805599453f;
// The running maximum may lag the true one by this many powers of two before
// the accumulators are rescaled: fp32 sums have room for it, and most tiles
// then skip the rescale.
constexpr float LAG = 8.0f;

// Zeros that the loads of keys outside the cache read instead.
static __device__ const uint4 attn_zero = {0, 0, 0, 0};

__device__ __forceinline__ uint32_t fdiv(uint32_t t, const FastDiv& f) {
  return __umulhi(2u * t, f.mul) >> f.shift;
}

// One 16-byte piece per lane from global memory into LDS: lane l's piece lands
// at lds + 16 l.  Written as assembly because the compiler would otherwise make
// every later LDS read wait for all of them; it has no register output, and
// the kernels wait with dma_wait before they read.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is reserved: declaring it is the point
__device__ __forceinline__ void dma16(const void* g, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(lds), "v"(g)
               : "memory", "m0");
}
// The same with a uniform base and a byte offset per lane.
__device__ __forceinline__ void dma16(const char* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
#pragma clang diagnostic pop
// Waits until at most N of the wave's vector-memory operations are in flight.
template <int N> __device__ __forceinline__ void dma_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
// Every LDS read issued so far has returned.
__device__ __forceinline__ void lds_wait() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }

// All waves of the workgroup come here, each with at most N vector-memory operations in
// flight and no LDS read; LDS accesses stay on their side.
template <int N> __device__ __forceinline__ void tile_barrier() {
  dma_wait<N>();
  lds_wait();
  __builtin_amdgcn_s_barrier();
  asm volatile("" : : : "memory");
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

__device__ __forceinline__ u32x4v_t lds_read16(uint32_t at) {
  return *(__attribute__((address_space(3))) const u32x4v_t*)(uintptr_t)at;
}

__device__ __forceinline__ float lds_read4(uint32_t at) {
  return *(__attribute__((address_space(3))) const float*)(uintptr_t)at;
}

// The four 16-bit values of this lane's column: within 16 lanes, lane i points
// at 4 elements of row i / 4 (columns 4 (i % 4) ..) and receives column i of the
// 4 x 16 block.
__device__ __forceinline__ s16x4_t lds_read_tr(uint32_t at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4_t*)(uintptr_t)at);
}

// 16-bit operand types of the matrix instructions.
template <typename E> struct Half;
template <> struct Half<bf16> {
  typedef bf16x8_t frag;
  typedef bf16x4_t quad;
  static constexpr float P_BIAS = 0.0f;
  static __device__ __forceinline__ f32x4_t mma16(frag a, frag b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16_t mma32(frag a, frag b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4_t mma16k16(s16x4_t a, quad b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(a, __builtin_bit_cast(s16x4_t, b), c, 0, 0, 0);
  }
  template <typename V> static __device__ __forceinline__ void set(V& f, int j, float x) {
    f[j] = (__bf16)x;
  }
  static __device__ __forceinline__ float widen(uint32_t bits) { return __uint_as_float(bits << 16); }
};
template <> struct Half<_Float16> {
  typedef f16x8_t frag;
  typedef _Float16 quad __attribute__((ext_vector_type(4)));
  // Probabilities are scaled by 2^6 so that small ones stay normal numbers of
  // fp16 (the largest is 2^(6 + LAG), well inside its range).
  static constexpr float P_BIAS = 6.0f;
  static __device__ __forceinline__ f32x4_t mma16(frag a, frag b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16_t mma32(frag a, frag b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4_t mma16k16(s16x4_t a, quad b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(quad, a), b, c, 0, 0, 0);
  }
  template <typename V> static __device__ __forceinline__ void set(V& f, int j, float x) {
    f[j] = (_Float16)x;
  }
  static __device__ __forceinline__ float widen(uint32_t bits) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  }
};

// The request and row tile of a workgroup.  Request i's tiles start at index
// floor(cu[i] G / ROWS) + i, which leaves it at least ceil(len G / ROWS) of them,
// so the grid needs no host knowledge of the lengths; tiles past a request's
// last row are empty.
struct RowTile {
  int req, start, len, seq;  // request, its first token row, token count and length
  int first, rows;           // first row of the tile, rows of the request
};
template <int ROWS>
__device__ __forceinline__ RowTile find_tile(const AttnLaunch& a, int tile, int lane) {
  RowTile t;
  if (a.n < 64) {
    // one round trip: lane i reads request i
    const int i = min(lane, a.n - 1);
    const int c = min(max(a.cu[i], 0), a.total);
    const int last = min(max(a.cu[a.n], 0), a.total), seq = a.seq[i];
    t.req = __popcll(__ballot(lane == 0 || (lane < a.n && c * a.group / ROWS + lane <= tile))) - 1;
    t.start = __builtin_amdgcn_readlane(c, t.req);
    const int end = t.req + 1 < a.n ? __builtin_amdgcn_readlane(c, t.req + 1) : last;
    t.len = max(end, t.start) - t.start;
    t.seq = max(__builtin_amdgcn_readlane(seq, t.req), 0);
  } else {
    int lo = 0, hi = a.n;
    while (hi - lo > 1) {
      const int step = (hi - lo + 63) / 64;
      const int i = lo + lane * step;
      bool in = lane == 0;
      if (!in && i < hi) {
        const int c = min(max(a.cu[i], 0), a.total);
        in = c * a.group / ROWS + i <= tile;
      }
      const int k = __popcll(__ballot(in)) - 1;
      lo += k * step;
      hi = min(hi, lo + step);
    }
    t.req = lo;
    t.start = min(max(a.cu[lo], 0), a.total);
    t.len = min(max(a.cu[lo + 1], t.start), a.total) - t.start;
    t.seq = max(a.seq[lo], 0);
  }
  t.rows = t.len * a.group;
  t.first = (tile - (t.start * a.group / ROWS + t.req)) * ROWS;
  if (t.first < 0) t.rows = 0;  // offsets that decrease: no rows rather than wrong ones
  return t;
}

// The whole request as one tile to start from.
__device__ __forceinline__ RowTile request_tile(const AttnLaunch& a, int req) {
  RowTile t;
  t.req = req;
  t.start = min(max(a.cu[req], 0), a.total);
  t.len = min(max(a.cu[req + 1], t.start), a.total) - t.start;
  t.seq = max(a.seq[req], 0);
  t.rows = t.len * a.group;
  t.first = 0;
  return t;
}

// The key tiles that a row tile with positions pa .. pb visits: those of the
// sinks [0, sink_end), then those of [lo, end).
template <int KT> struct KeyRange {
  int lo, end, sink_end;
  int n1, skip, tiles;  // tiles before the gap, tiles in the gap, tiles visited
  __device__ __forceinline__ KeyRange(const AttnLaunch& a, int pa, int pb, int seq) {
    end = max(0, min(min(pb + 1, seq), (int)a.key_capacity));
    lo = a.window > 0 ? max(0, max(0, pa) - a.window + 1) : 0;
    lo = min(lo, end);
    sink_end = min(a.sinks, lo);
    n1 = (sink_end + KT - 1) / KT;
    const int w0 = max(n1, lo / KT);
    skip = w0 - n1;
    tiles = max(n1, (end + KT - 1) / KT - skip);
    if (end == 0) tiles = 0;
  }
  __device__ __forceinline__ int base(int i) const { return KT * (i < n1 ? i : i + skip); }
  __device__ __forceinline__ bool has(int t) const { return t < end && (t >= lo || t < sink_end); }
};

// Splits of a visit of `tiles` key tiles: at most `splits`, of at least `least` tiles
// each; per = tiles of one split.
__device__ __forceinline__ int split_of(int tiles, int splits, int least, int& per) {
  const int n = max(1, min(splits, tiles / least));
  per = (tiles + n - 1) / n;
  return max(1, (tiles + max(per, 1) - 1) / max(per, 1));
}

// 64 consecutive entries of one block table row, one per lane.  Everything but `entry`
// is wave-uniform.
struct PageWindow {
  const int32_t* row;
  int base, entry;
  int first_key, end_key;  // the keys of its pages
  uint64_t none;           // lanes without a page
  __device__ __forceinline__ PageWindow(const AttnLaunch& a, int req)
      : row(a.table + (int64_t)req * a.table_stride), base(0), entry(-1), first_key(0), end_key(0),
        none(0) {}
  // Makes the pages of the keys first .. last available (at most 64 of them).
  __device__ __forceinline__ void cover(const AttnLaunch& a, int first, int last, int lane) {
    if (first >= first_key && last < end_key) return;
    base = (int)fdiv(first, a.page);
    const int i = base + lane;
    const int e = i < a.max_pages ? row[i] : -1;
    entry = (uint32_t)e < (uint32_t)a.num_pages ? e : -1;
    none = __ballot(entry < 0);
    first_key = base * (int)a.page.d;
    end_key = (int)min((int64_t)(base + 64) * a.page.d, (int64_t)INT32_MAX);
  }
  // Whether any of the keys first .. last lies on no page.
  __device__ __forceinline__ bool missing(const AttnLaunch& a, int first, int last) const {
    if (none == 0) return false;
    const int p0 = (int)fdiv(first, a.page), p1 = (int)fdiv(last, a.page);
    return (none >> (p0 - base)) & (~0ull >> (63 - (p1 - p0)));
  }
  // The page at index `page` of the row (a lane's own, or a uniform one), -1 if none.  All
  // lanes have to ask, with or without a use for it: one that is switched off hands out
  // page 0 in place of its entry.
  __device__ __forceinline__ int at(int page) const {
    return __builtin_amdgcn_ds_bpermute(4 * (page - base), entry);
  }
  __device__ __forceinline__ int uniform_at(int page) const {
    return __builtin_amdgcn_readlane(entry, page - base);
  }
};

// Bits 0 .. n (none for n < 0) of a word.
__device__ __forceinline__ uint32_t bits_to(int n) {
  return n < 0 ? 0u : n >= 31 ? ~0u : (2u << n) - 1u;
}
// The keys base .. base + 31 that a row at position pos sees, as bits, of those in
// `there`.
__device__ __forceinline__ uint32_t seen(const AttnLaunch& a, int base, int pos, uint32_t there) {
  uint32_t s = there & bits_to(pos - base);
  if (a.window > 0) s &= ~bits_to(pos - a.window - base) | bits_to(a.sinks - 1 - base);
  return s;
}

__device__ __forceinline__ int wave_of() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Max / sum over the lanes l, l ^ 32.
__device__ __forceinline__ float max_half(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_half(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Max / sum over the lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float max_quarter(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return max_half(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float sum_quarter(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return sum_half(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

}  // namespace kda
