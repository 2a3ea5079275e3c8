// Paged attention of few rows per request over a cache in 8 bits (decode, short drafts).
//
// The one-pass softmax of the 16-bit rows kernel: a workgroup of four waves holds 16 or 32
// rows of one kv head, each wave walks its own quarter of the keys, and the four are joined
// through LDS at the end.  Codes come by DMA into each wave's own part of LDS as they are, 32
// keys at a time with their scales, and are widened in registers right before the matrix
// instructions, once for all rows:
//
//   scores   a lane's 16 bytes are 16 channels of one key: two fragments, widened with the
//            key's scale (a power of two, so the values are exact in bf16)
//   values   the transposing 8-byte read gives a lane 8 keys of one channel; the keys'
//            scales go into the probabilities, which become bf16 (whatever the rows' type: it has
//            the range that a scale may ask for), as a pair where that is free or needed
//
// Bound by HBM: a key's codes are 256 bytes for 128 channels, half of the 16-bit cache's, and are
// read once for all rows of the tile.  256 ragged decode requests (0.86 GB of codes): 166 to 171
// us, 5.0 to 5.2 TB/s (with even lengths of 4096 keys 5.4), where a large copy reaches 5.2 and a
// plain read 6.3.  The same DMA with nothing computed takes 2 to 4 % less, so what is left is the
// ragged end and the start of a short stream.  One buffer each for K and V, refilled as soon as it
// is read, leaves room for four workgroups on a compute unit; a double buffer and two workgroups
// take the same time, as do all heads of a piece on one XCD.  With 32 rows two workgroups fit, fewer
// bytes are on their way (1.5 waves a SIMD in place of 2.7), and the same keys take longer: 256 requests of
// 8 tokens 248 us in e4m3 and 270 in int8, of 4 tokens (16 rows) 201.
#include "kda_attn_q8.hpp"

namespace kda {
namespace {

constexpr int WAVES = 4, KT = 32;  // keys per tile

// Piece p of row r of a tile sits in slot p ^ swz(r) of the row.  K is read one piece each of
// 16 rows, V 16 bytes of the rows 0..7 and 16..23 (or 8..15 and 24..31) at a time: either
// spreads over the 256 bytes of all banks.
template <int P> __device__ __forceinline__ int kswz(int r) { return P == 8 ? (r >> 1) & 7 : (r >> 2) & 3; }
template <int P> __device__ __forceinline__ int vswz(int r) {
  return P == 8 ? ((r >> 1) & 3) | ((r >> 2) & 4) : ((r >> 2) & 1) | ((r >> 3) & 2);
}

// Four bytes per lane from global memory into LDS: lane l's land at lds + 4 l.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is reserved: declaring it is the point
__device__ __forceinline__ void dma4(const void* g, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(lds), "v"(g)
               : "memory", "m0");
}
#pragma clang diagnostic pop

__device__ __forceinline__ u32x2v_t lds_read_tr8(uint32_t at) {
  typedef int i32x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(u32x2v_t, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
      (__attribute__((address_space(3))) i32x2_t*)(uintptr_t)at));
}

// A NaN code of V spoils the product of its tile also for rows that do not see its key (0 times
// NaN).  Where a sum is not finite, the keys are gone through twice more: once with NaN codes
// as ones and the others as zeros, each visible key weighing one, which finds the sums that a NaN
// belongs to, and once with zeros for NaN.  The counts are never rescaled: a maximum that grows by
// 2^150 would make them 0, where the NaN itself stays.
enum { PLAIN = 0, COUNT = 1, ZEROED = 2 };
__device__ __forceinline__ uint32_t without_nan(uint32_t w, int mode) {
  const uint32_t nan = (((w & 0x7f7f7f7fu) + 0x01010101u) >> 7 & 0x01010101u) * 0xffu;  // bytes 0x7f, 0xff
  return mode == COUNT ? nan & 0x38383838u : w & ~nan;                                   // (0x38 is 1)
}

struct Tile {
  int base;        // its first key
  uint32_t valid;  // which of its keys exist
};

template <typename E, int DIM, int RB, int CODE>
__global__ __launch_bounds__(256, RB == 1 ? 4 : 2) void rows_q8_kernel(const AttnQ8Launch a) {
  typedef typename Half<E>::frag frag;
  constexpr uint32_t ALL = ~0u;
  // Probabilities as a pair of bf16: 16 bits.  With 16 rows the second product is free (256 requests of
  // 64 .. 8192 keys: 179 us with and without), with 32 it takes time (8 tokens each: 264 us, 248 us
  // without), and rows in fp16 need its bits.
  constexpr bool PAIR = RB == 1 || std::is_same_v<E, _Float16>;
  constexpr int P = DIM / 16;                    // 16-byte pieces per row
  constexpr int NI = KT * P / 64;                // DMA instructions per K or V tile
  constexpr int QS = DIM / 32;                   // fragments of a row
  constexpr int STAGE = 2 * KT * P + 32;         // pieces of a K and a V tile, and two tiles' scales
  constexpr int ROWS = 64 / P, ROW = DIM;        // keys of a DMA instruction, bytes of one
  constexpr int OS = DIM + 4;                    // floats per joined row (padded)
  constexpr int JOIN = WAVES * 16 * RB * OS / 4;
  constexpr int PIECES = WAVES * STAGE > JOIN ? WAVES * STAGE : JOIN;
  __shared__ __attribute__((aligned(1024))) uint4 smem[PIECES];
  __shared__ float sm_m[WAVES][16 * RB], sm_l[WAVES][16 * RB];

  const int lane = threadIdx.x & 63, wave = wave_of();
  const int l16 = lane & 15, gq = lane >> 4;
  // heads fastest, so that neighbouring workgroups share pages of the table and lines of the scales
  const uint32_t unit = fdiv(blockIdx.x, a.hdiv);
  const int kvh = (int)(blockIdx.x - unit * a.hkv), split = blockIdx.y;
  const RowTile rt = request_tile(a, (int)unit);
  if (rt.rows == 0) return;
  const int seq = rt.seq, pos0 = seq - rt.len;
  const float c = a.scale * LOG2E;
  uint4* const my = smem + wave * STAGE;
  // this lane's piece of an instruction's keys, as bytes from the first of them
  const uint32_t koff = lane / P * ROW + 16 * (lane % P ^ kswz<P>(lane / P));
  const uint32_t voff = lane / P * ROW + 16 * (lane % P ^ vswz<P>(lane / P));
  // LDS byte addresses of fragments in the first stage.  K: key 16 k + l16, piece 4 i + gq.  V:
  // what this lane points the transposing reads at, 8 bytes of piece d of key vrow, so
  // that it receives channel 16 d + l16 of the keys 4 gq + 0..3 and 16 + 4 gq + 0..3.
  const uint32_t ka = lds_addr(my + l16 * P + (gq ^ kswz<P>(l16)));
  const int vrow = 4 * gq + ((l16 >> 1) & 3) + 16 * (l16 >> 3);
  const uint32_t va = lds_addr(my + KT * P + vrow * P + vswz<P>(vrow)) + 8 * (l16 & 1);
  const uint32_t sa = lds_addr(my + 2 * KT * P);  // scales of K, then of V; 256 bytes on, the other tile's
  const bool even = a.page.d % ROWS == 0;         // whether an instruction's keys share a page
  PageWindow pages(a, rt.req);
  const char* const kbase = (const char*)a.kc + (int64_t)kvh * a.page.d * ROW;
  const char* const vbase = (const char*)a.vc + (int64_t)kvh * a.page.d * ROW;
  const int64_t scale_page = (int64_t)a.hkv * a.scales.per_page;

  // One tile of rows, and the further ones of a request that has more than its hint said.
  for (int first = rt.first; first < rt.rows; first += 16 * RB) {
    const int rows = min(16 * RB, rt.rows - first);
    const int pa = pos0 + (int)fdiv(first, a.gdiv);
    const int pb = pos0 + (int)fdiv(first + rows - 1, a.gdiv);
    const KeyRange<KT> range(a, pa, pb, seq);
    int per;
    const int splits = split_of(range.tiles, a.splits, a.min_keys / KT, per);
    if (split >= splits) continue;
    const int t0 = split * per, nt = max(0, min(per, range.tiles - t0));

    // this lane's rows (the MFMA columns l16 of each block): their queries, zero past the last
    // row, in the order of the keys' channels, and their positions
    u32x4v_t q[RB][QS];
    int qpos[RB];
    int ql = lane;
    asm volatile("" : "+v"(ql));  // or what follows would be kept through the walk
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int r = 16 * b + (ql & 15), gq = ql >> 4;
      const int tok = (int)fdiv(first + r, a.gdiv);
      const int head = kvh * a.group + first + r - tok * a.group;
      qpos[b] = pos0 + tok;
      const bool in = r < rows;
      const u32x4v_t* src = reinterpret_cast<const u32x4v_t*>(
          (const E*)a.q + (in ? (int64_t)(rt.start + tok) * a.q_stride + head * DIM : 0));
#pragma unroll
      for (int s = 0; s < QS; ++s) q[b][s] = in ? src[8 * (s / 2) + 2 * gq + s % 2] : u32x4v_t{0, 0, 0, 0};
    }

    f32x4_t o[DIM / 16][RB];
    float m[RB], l[RB];

    // Where key tile i starts and which of its keys exist.
    auto locate = [&](int i) __attribute__((always_inline)) {
      Tile t;
      t.base = range.base(i);
      const int last = min(t.base + KT - 1, (int)a.key_capacity - 1);
      pages.cover(a, t.base, last, lane);
      // inside the range and with every page there (the common case), all keys exist
      t.valid = ALL;
      if (t.base + KT > range.end || !(t.base >= range.lo || t.base + KT <= range.sink_end) ||
          pages.missing(a, t.base, last)) {
        const int key = t.base + (lane & (KT - 1));
        const int page = pages.at((int)fdiv(key, a.page));  // of every lane's key
        t.valid = (uint32_t)__ballot(range.has(key) && page >= 0);
      }
      return t;
    };
    // Issues the DMA of its K codes and of its scales, or of its V codes.
    auto issue_scales = [&](const Tile& t, int slot) __attribute__((always_inline)) {
      // lane l: K's scale of key l % 32, or V's
      int ln = lane;
      asm volatile("" : "+v"(ln));  // or the pool's address would be kept
      const float* const scales = (ln < KT ? a.scales.k : a.scales.v) + (int64_t)kvh * a.scales.per_page;
      const int r = ln & (KT - 1), key = t.base + r, pg = (int)fdiv(key, a.page);
      const int64_t page = pages.at(pg);
      const float* p = scales + page * scale_page + fdiv(key - pg * (int)a.page.d, a.scales.block);
      if (!((t.valid >> r) & 1)) p = (const float*)&attn_zero;
      dma4(p, lds_addr(my + 2 * KT * P + 16 * slot));
    };
    auto issue = [&](const Tile& t, bool v) __attribute__((always_inline)) {
      uint4* const to = v ? my + KT * P : my;
      const char* const pool = v ? vbase : kbase;
      const int64_t stride = v ? a.v_page : a.k_page;
      if (even && t.valid == ALL) {
        // one page per instruction: the addresses are scalar work
        uint32_t o = v ? voff : koff;
        asm volatile("" : "+v"(o));  // or every x would keep its register
#pragma unroll
        for (int x = 0; x < NI; ++x) {
          const int key = t.base + x * ROWS, pg = (int)fdiv(key, a.page);
          const int64_t off = key - pg * (int)a.page.d, page = pages.uniform_at(pg);
          // (the swizzles are linear: that of row r0 + x ROWS is r0's xor that of x ROWS)
          dma16(pool + page * stride + off * ROW, o ^ 16 * (v ? vswz<P>(x * ROWS) : kswz<P>(x * ROWS)),
                lds_addr(to + 64 * x));
        }
        return;
      }
#pragma unroll 1
      for (int x = 0; x < NI; ++x) {
        const int r = (64 * x + lane) / P, ps = lane % P, key = t.base + r;
        const int pg = (int)fdiv(key, a.page);
        const int64_t off = key - pg * (int)a.page.d, page = pages.at(pg);
        const char* p = pool + page * stride + off * ROW + 16 * (ps ^ (v ? vswz<P>(r) : kswz<P>(r)));
        if (!((t.valid >> r) & 1)) p = (const char*)&attn_zero;
        dma16(p, lds_addr(to + 64 * x));
      }
    };

    f32x4_t s[2][RB];
    auto scores = [&](int slot) __attribute__((always_inline)) {  // S^T = K Q^T
      uint32_t at = ka;
      asm volatile("" : "+v"(at));  // or every step would keep its address
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float sk = lds_read4(sa + 256 * slot + 64 * k + 4 * l16);
        if constexpr (CODE == INT8) sk = pow2_scale(sk);
#pragma unroll
        for (int b = 0; b < RB; ++b) s[k][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < P / 4; ++i) {
          const u32x4v_t w = lds_read16((at + k * 16 * ROW) ^ 64 * i);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const u32x2v_t lo = Code<CODE>::widen16(E{}, w[2 * y], sk), hi = Code<CODE>::widen16(E{}, w[2 * y + 1], sk);
            const frag kf = __builtin_bit_cast(frag, u32x4v_t{lo[0], lo[1], hi[0], hi[1]});
#pragma unroll
            for (int b = 0; b < RB; ++b)
              s[k][b] = Half<E>::mma16(kf, __builtin_bit_cast(frag, q[b][2 * i + y]), s[k][b]);
          }
        }
      }
    };
    // The softmax of the tile's scores, and its product with V once `values` says that it is there.
    auto weigh = [&](int mode, const Tile& t, int slot, auto values) __attribute__((always_inline)) {
      // keys hidden from some rows, or absent
      const bool mixed = pa != pb && (t.base + KT - 1 > pa ||
                                      (a.window > 0 && t.base <= pb - a.window && t.base + KT > a.sinks));
      if (mixed || t.valid != ALL) {
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          const uint32_t see = seen(a, t.base, qpos[b], t.valid) >> (4 * gq);
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r) s[k][b][r] = see & (1u << (16 * k + r)) ? s[k][b][r] : NEG_INF;
        }
      }
      // softmax: the maximum over the tile's keys, the rescale where it grew by
      // more than LAG, the probabilities
      float mx[RB];
      bool grew = false;
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        float x = NEG_INF;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int r = 0; r < 4; ++r) x = fmaxf(x, s[k][b][r]);
        mx[b] = max_quarter(x) * c;  // c > 0
        grew |= mx[b] > m[b] + LAG;
      }
      if (!(CODE == E4M3 && mode == COUNT) && __any(grew)) {
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          const float nm = fmaxf(m[b], mx[b]);
          const float f = nm == NEG_INF ? 1.0f : exp2_fast(m[b] - nm);
          m[b] = nm;
          l[b] *= f;
#pragma unroll
          for (int d = 0; d < DIM / 16; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) o[d][b][r] *= f;
        }
      }
      // the probabilities, times V's scales
      const uint32_t sv = sa + 256 * slot + 4 * KT + 16 * gq;
      f32x4_t vs[2];
      vs[0] = __builtin_bit_cast(f32x4_t, lds_read16(sv));
      vs[1] = __builtin_bit_cast(f32x4_t, lds_read16(sv + 64));
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        // a row that has seen no key yet keeps m = -inf: its scores are all -inf too
        const float mb = m[b] == NEG_INF ? 0.0f : m[b];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float p = exp2_fast(fmaf(s[k][b][r], c, -mb));
            l[b] += p;
            s[k][b][r] = p;
          }
      }
      if (mixed) {  // a hidden key has no weight, whatever its scale
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) s[k][b][r] = s[k][b][r] == 0.0f ? 0.0f : s[k][b][r] * pow2_scale(vs[k][r]);
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) s[k][b][r] *= pow2_scale(vs[k][r]);
      }
      values();
      if (CODE == E4M3 && mode != PLAIN) {
#pragma unroll 1
        for (int x = 0; x < NI; ++x) {
          uint4* const at = my + KT * P + 64 * x + lane;
          const uint4 u = *at;
          *at = make_uint4(without_nan(u.x, mode), without_nan(u.y, mode), without_nan(u.z, mode),
                           without_nan(u.w, mode));
        }
        lds_wait();
      }
      if (CODE == E4M3 && mode == COUNT) {
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          const uint32_t see = seen(a, t.base, qpos[b], t.valid) >> (4 * gq);
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r) s[k][b][r] = see & (1u << (16 * k + r)) ? 1.0f : 0.0f;
        }
      }
      // P^T as it lies: lane group gq holds keys 4 gq + r and 16 + 4 gq + r
      bf16x8_t p[RB], pl[RB];
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = s[j / 4][b][j % 4];
          p[b][j] = (__bf16)x;
          if constexpr (PAIR) pl[b][j] = (__bf16)(x - (float)p[b][j]);
        }
      uint32_t at = va;
      asm volatile("" : "+v"(at));
      float one = 1.0f;
      if constexpr (CODE == INT8) asm volatile("" : "+v"(one));  // or bytes go through integers
#pragma unroll
      for (int d = 0; d < DIM / 16; ++d) {
        if (d % 4 == 0) __builtin_amdgcn_sched_barrier(0);  // few registers at a time
        const u32x2v_t w = lds_read_tr8(at ^ 16 * d);
        const u32x2v_t lo = Code<CODE>::widen16(bf16{}, w[0], one), hi = Code<CODE>::widen16(bf16{}, w[1], one);
        const bf16x8_t v = __builtin_bit_cast(bf16x8_t, u32x4v_t{lo[0], lo[1], hi[0], hi[1]});
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          o[d][b] = Half<bf16>::mma16(v, p[b], o[d][b]);
          if constexpr (PAIR) o[d][b] = Half<bf16>::mma16(v, pl[b], o[d][b]);
        }
      }
    };

    // contiguous tiles per wave
    const int share = (nt + WAVES - 1) / WAVES;
    const int w0 = t0 + min(nt, wave * share), w1 = t0 + min(nt, (wave + 1) * share);
    auto walk = [&](int mode) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        m[b] = NEG_INF;
        l[b] = 0.0f;
#pragma unroll
        for (int d = 0; d < DIM / 16; ++d) o[d][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
      if (w0 >= w1) return;
      // one buffer each for K and V, refilled as soon as it is read
      Tile cur = locate(w0);
      issue_scales(cur, 0);
      issue(cur, false);
      issue(cur, true);
      // the queries arrive here: a wait for them in the loop would wait for the DMA too
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int x = 0; x < QS; ++x) asm volatile("" : "+v"(q[b][x]));
#pragma unroll 1
      for (int i = w0; i < w1; ++i) {
        const bool more = i + 1 < w1;
        const int slot = (i - w0) & 1;
        Tile next = cur;
        dma_wait<NI>();  // K and the scales of this tile; V may still be on its way
        scores(slot);
        lds_wait();
        if (more) {
          next = locate(i + 1);
          issue_scales(next, slot ^ 1);
          issue(next, false);
        }
        weigh(mode, cur, slot, [&] {
          if (more) dma_wait<NI + 1>();
          else dma_wait<0>();
        });
        lds_wait();
        if (more) issue(next, true);
        cur = next;
      }
    };
    uint32_t nan_at[RB] = {};  // sums that a NaN belongs to, a bit each
    for (int mode = PLAIN;;) {
      walk(mode);
      // int8 has no NaN, and with one position every key of a tile is visible to all rows
      if (CODE != E4M3 || pa == pb || mode == ZEROED) break;
      if (mode == PLAIN) {
        float z = 0.0f;  // becomes NaN if any sum is not finite
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int d = 0; d < DIM / 16; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) z = fmaf(o[d][b][r], 0.0f, z);
        if (!__any(z != 0.0f)) break;
        mode = COUNT;
      } else {
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int d = 0; d < DIM / 16; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              nan_at[b] |= o[d][b][r] > 0.0f ? 1u << (4 * d + r) : 0u;
        mode = ZEROED;
      }
      lds_wait();
    }
    if constexpr (CODE == E4M3) {
#pragma unroll
      for (int b = 0; b < RB; ++b)
        if (__any(nan_at[b] != 0)) {
#pragma unroll
          for (int d = 0; d < DIM / 16; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (nan_at[b] >> (4 * d + r) & 1) o[d][b][r] = __builtin_nanf("");
        }
    }

    // join of the four waves (the thread's place worked out here, not kept through the walk)
    int jl = lane;
    asm volatile("" : "+v"(jl));
    const int jq = jl >> 4, tid = jl + 64 * wave;
    jl &= 15;
#pragma unroll
    for (int b = 0; b < RB; ++b) l[b] = sum_quarter(l[b]);
    __syncthreads();
    float* const so = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int r = 16 * b + jl;
      if (jq == 0) {
        sm_m[wave][r] = m[b];
        sm_l[wave][r] = l[b];
      }
#pragma unroll
      for (int d = 0; d < DIM / 16; ++d)
        *reinterpret_cast<f32x4_t*>(so + (wave * 16 * RB + r) * OS + 16 * d + 4 * jq) = o[d][b];
    }
    __syncthreads();
    constexpr int PER = DIM / 4;  // threads per row
    for (int x = tid; x < rows * PER; x += 64 * WAVES) {
      const int r = x / PER, d = 4 * (x % PER);
      float top = sm_m[0][r];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) top = fmaxf(top, sm_m[w][r]);
      const float base = top == NEG_INF ? 0.0f : top;
      float sum = 0.0f;
      f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const float f = exp2_fast(sm_m[w][r] - base);
        sum = fmaf(f, sm_l[w][r], sum);
        const f32x4_t y = *reinterpret_cast<const f32x4_t*>(so + (w * 16 * RB + r) * OS + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(f, y[i], acc[i]);
      }
      // a row that sees no key has sum 0: zeros, and a log-sum-exp of -inf
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = sum == 0.0f ? 0.0f : acc[i] * inv;
      const float lse2 = sum == 0.0f ? NEG_INF : base + __log2f(sum);
      const int tok = (int)fdiv(first + r, a.gdiv);
      const int head = kvh * a.group + first + r - tok * a.group;
      const int64_t row = (int64_t)(rt.start + tok) * a.hq + head;
      if (a.part_n != nullptr && split == 0 && d == 0) a.part_n[row] = splits;
      if (splits == 1) {
        store4((E*)a.out + row * DIM + d, acc[0], acc[1], acc[2], acc[3]);
        if (a.lse != nullptr && d == 0) a.lse[row] = lse2 * LN2;
      } else {
        const int64_t prow = (int64_t)split * a.total * a.hq + row;
        store4(a.part_o + prow * DIM + d, acc[0], acc[1], acc[2], acc[3]);
        if (d == 0) a.part_lse[prow] = lse2;
      }
    }
    __syncthreads();  // before the next tile's DMA
  }
}

template <typename E, int DIM, int RB, int CODE> hipError_t rows_go(const AttnQ8Launch& L) {
  hipLaunchKernelGGL((rows_q8_kernel<E, DIM, RB, CODE>), dim3((unsigned)(L.n * L.hkv), (unsigned)L.splits),
                     dim3(64 * WAVES), 0, (hipStream_t)L.stream, L);
  return hipGetLastError();
}
template <typename E, int DIM, int RB> hipError_t rows_code(const AttnQ8Launch& L) {
  return L.code == E4M3 ? rows_go<E, DIM, RB, E4M3>(L) : rows_go<E, DIM, RB, INT8>(L);
}
template <typename E, int DIM> hipError_t rows_rb(const AttnQ8Launch& L) {
  return L.row_blocks == 1 ? rows_code<E, DIM, 1>(L) : rows_code<E, DIM, 2>(L);
}
template <typename E> hipError_t rows_dim(const AttnQ8Launch& L) {
  return L.dim == 64 ? rows_rb<E, 64>(L) : rows_rb<E, 128>(L);
}

}  // namespace

hipError_t launch_attn_q8_rows(const AttnQ8Launch& L) {
  return L.dtype == 1 ? rows_dim<bf16>(L) : rows_dim<_Float16>(L);
}

}  // namespace kda
