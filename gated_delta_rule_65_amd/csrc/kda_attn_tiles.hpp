// Paged attention of long chunks of new tokens (bf16, fp16), over a cache of that type or in
// 8 bits: the kernel that both instantiate.
//
// The same one-pass softmax as the rows kernel, with the work of a matrix product:
// a workgroup holds 32 rows per wave and all its waves walk the keys together, 64
// at a time, from K and V tiles in LDS.  S^T = K Q^T and O^T = V^T P^T run on
// 32 x 32 x 16 matrix instructions; lane l holds row l % 32 of its wave, in S^T as in
// O^T, so a row's maximum and sum take one swap between the wave's halves.
//
// Bound by the matrix cores and the vector unit together: a tile of 64 keys costs a
// wave 32 products (1024 cycles for 128 channels) and about 100 vector instructions
// beside 32 exponentials (nearly as much), and a SIMD holds two waves (256 registers).
// So the two have to be out of step, one multiplying while the other weighs.  They
// drift apart by themselves where barriers are rare; products go first (s_setprio).
// 2048 tokens on 131072 keys, 32 heads on 8, takes 3.7 to 3.95 ms from card to card (1.18
// to 1.10 PFLOP/s, matrix cores 55 % busy; a large library product reaches 1.23).  Measured
// on the way, same case, one card:
//   a barrier a tile, both waves in step                          4.26 ms
//   the phases of the two waves held apart by barriers            4.46 ms
//   a tile's products woven into the softmax of the one before    4.60 ms
//   two tiles a barrier                                           4.06 ms
//   the same, products first                                      3.93 ms
//   the same, fragment addresses constant within a ring half      3.82 ms
// Fragment reads stay three ahead of their products: left to the compiler each product
// waits for its own read (5.87 ms, with the phases held apart).
//
// Both shapes have two waves per SIMD and 128 KB of LDS per compute unit.  Eight waves
// (256 rows, two tiles a barrier) read each key half as often, which long visits need;
// two workgroups of four waves (128 rows, a tile a barrier) even out ragged requests
// (33 requests of 1 .. 700 tokens: 157 us against 184 us; 2048 tokens on 131072 keys:
// 4.54 ms against 3.93 ms, both without splits).
//
// Over a cache in 8 bits the products are the same: each tile's codes are widened once for the
// workgroup's rows, with their scales, into the tile in LDS that a 16-bit cache's DMA would fill.
// 2048 tokens on 131072 keys, 32 heads on 8, take 3.90 to 4.39 ms in e4m3 from card to card, and 2 to 3 %
// more in int8 (4.03 beside 3.95: nine instructions for four int8 codes, two for four of e4m3).
// That is 5 to 8 % more than in 16 bits on the same card: the conversions and addresses are vector and scalar work of
// the same waves (without either: 3.5 ms).  Measured on the way, e4m3:
//   codes fetched and widened at the end of two tiles, by flat loads          4.74 ms
//   by global loads (every LDS read waits for a flat load)                    4.59 ms
//   fragment reads and products in an order spelled out                       4.18 ms
//   one tile's codes in registers, widened among the scores' products,
//   fetched among the values'                                                 4.08 ms
//   the fetch without branches                                                4.05 ms
//   nothing to spread the writes over all banks, writes two products later    3.96 ms
#pragma once
#include "kda_attn_q8.hpp"

namespace kda {
namespace {

constexpr int KT = 64;    // keys per tile
constexpr int MFMA = 0x8, DS_READ = 0x100;  // instruction classes of sched_group_barrier

// A fragment read takes one piece each of 16 consecutive rows at a time: they spread
// over the 256 bytes of all banks.
template <int P> __device__ __forceinline__ int kswz(int r) { return P == 16 ? r & 15 : (r >> 1) & 7; }
// The transposing read takes 32 bytes of rows r .. r + 3 at two neighbouring
// 32-byte columns per half wave: with this the eight fall into different banks.
template <int P> __device__ __forceinline__ int vswz(int r) {
  return P == 16 ? 2 * (2 * (r & 3) + ((r >> 2) & 1)) : 2 * ((r & 2) | ((r >> 2) & 1));
}

// CODE: the codes of a cache in 8 bits (A is AttnQ8Launch), or NO_CODE.
constexpr int NO_CODE = -1;
template <typename A, typename E, int DIM, int NW, int CODE>
__global__ __launch_bounds__(64 * NW, CODE != NO_CODE && DIM == 64 ? 3 : 2) void tiles_kernel(const A a) {
  typedef typename Half<E>::frag frag;
  constexpr int P = DIM / 8;            // 16-byte pieces per row
  constexpr int NI = P / NW;            // DMA instructions per wave and tile, K or V
  constexpr int QS = DIM / 16, DV = DIM / 32;
  constexpr int RING = NW / 2, PAIR = RING / 2;  // tiles in LDS, tiles per barrier
  static_assert(P % NW == 0, "a tile splits evenly over the waves");
  __shared__ uint4 smem_k[RING][KT * P], smem_v[RING][KT * P];

  const int lane = threadIdx.x & 63, wave = wave_of();
  const int l32 = lane & 31, h = lane >> 5;
  // later tiles have more keys: they go first
  const uint32_t work = gridDim.x - 1 - blockIdx.x, unit = fdiv(work, a.hdiv);
  const int kvh = (int)(work - unit * a.hkv), split = blockIdx.y;
  const RowTile rt = find_tile<32 * NW>(a, (int)unit, lane);
  if (rt.first >= rt.rows || rt.rows == 0) return;
  const int rows = min(32 * NW, rt.rows - rt.first);
  const int seq = rt.seq, pos0 = seq - rt.len;
  const KeyRange<KT> range(a, pos0 + (int)fdiv(rt.first, a.gdiv),
                           pos0 + (int)fdiv(rt.first + rows - 1, a.gdiv), seq);
  int per;
  const int splits = split_of(range.tiles, a.splits, a.min_keys / KT, per);
  if (split >= splits) return;
  const int t0 = split * per, t1 = min(range.tiles, t0 + per);

  constexpr bool Q8 = CODE != NO_CODE;
  // Beside codes on their way there are no registers for what only the end needs: it is
  // worked out again there.
  struct Place {
    int tok, head;
    bool in;
  };
  auto place = [&](int ln) __attribute__((always_inline)) {
    const int r = 32 * wave + (ln & 31), tok = (int)fdiv(rt.first + r, a.gdiv);
    return Place{tok, kvh * a.group + rt.first + r - tok * a.group, r < rows};
  };
  auto again = [](int x) __attribute__((always_inline)) {
    if constexpr (Q8) asm volatile("" : "+v"(x));
    return x;
  };

  // this lane's row
  const int r = 32 * wave + l32;
  const bool in = r < rows;
  const int tok = (int)fdiv(rt.first + r, a.gdiv);
  const int head = kvh * a.group + rt.first + r - tok * a.group;
  const int qpos = pos0 + tok;
  // positions of the wave's first and last row
  const int wa = pos0 + (int)fdiv(rt.first + 32 * wave, a.gdiv);
  const int wb = pos0 + (int)fdiv(rt.first + min(32 * wave + 31, rows - 1), a.gdiv);
  // Where this lane's query row begins, as an element of q (-1 past the last row).
  const int64_t qrow = in ? (int64_t)(rt.start + tok) * a.q_stride + head * DIM : -1;
  frag q[QS];

  // LDS byte addresses of the fragments in stage 0: key row l32 of a K tile, and the
  // rows and columns that this lane points the transposing reads at (both swizzles
  // depend on the row modulo 16 alone, so the other rows are constants away)
  uint32_t ka[QS], va[DV];
#pragma unroll
  for (int x = 0; x < QS; ++x) ka[x] = lds_addr(&smem_k[0][l32 * P + ((2 * x + h) ^ kswz<P>(l32))]);
#pragma unroll
  for (int d = 0; d < DV; ++d) {
    const int i16 = lane & 15, row = 4 * h + (i16 >> 2);
    const int piece = 4 * d + 2 * ((lane >> 4) & 1) + ((i16 & 3) >> 1);
    va[d] = lds_addr(&smem_v[0][row * P + (piece ^ vswz<P>(row))]) + 8 * (i16 & 1);
  }
  constexpr int STAGE = KT * P * 16, ROW = P * 16;  // bytes

  f32x16_t o[DV];
  float m, l;
  const float c = a.scale * LOG2E;

  PageWindow pages(a, rt.req);
  const char* const kbase = (const char*)a.kc + (int64_t)kvh * a.page.d * (CODE == NO_CODE ? DIM * 2 : DIM);
  const char* const vbase = (const char*)a.vc + (int64_t)kvh * a.page.d * (CODE == NO_CODE ? DIM * 2 : DIM);

  // Byte offsets of this lane's pieces from the first of an instruction's keys (64 / P
  // of them; the swizzles depend on the row modulo 16 alone, which is the same for
  // every instruction of this wave), and whether those always share a page.
  const int lrow = (64 * wave + lane) / P, lps = lane % P;
  const uint32_t koff = lane / P * ROW + 16 * (lps ^ kswz<P>(lrow));
  const uint32_t voff = lane / P * ROW + 16 * (lps ^ vswz<P>(lrow));
  static_assert(NW * (64 / P) % 16 == 0, "a wave's rows agree modulo 16");
  const bool even = a.page.d % (64 / P) == 0;

  // The page that this wave's DMA is in: its first key, and where its rows of this
  // head begin (scalar values, kept from one instruction to the next).
  int page_key = -(1 << 30);
  const char *kpage = nullptr, *vpage = nullptr;

  // Makes the pages of the key tile at `base` available; returns which of its keys exist.
  auto locate = [&](int base) __attribute__((always_inline)) -> uint64_t {
    const int last = min(base + KT - 1, (int)a.key_capacity - 1);
    pages.cover(a, base, last, lane);
    // inside the range and with every page there (the common case), all keys exist
    uint64_t valid = ~0ull;
    if (base + KT > range.end || !(base >= range.lo || base + KT <= range.sink_end) ||
        pages.missing(a, base, last)) {
      const int key = base + lane;
      const int page = pages.at((int)fdiv(key, a.page));  // of every lane's key
      valid = __ballot(range.has(key) && page >= 0);
    }
    return valid;
  };
  // Issues the DMA of the key tile at `base`; returns which of its keys exist.
  auto issue = [&](int base, int stage) __attribute__((always_inline)) -> uint64_t {
    const uint64_t valid = locate(base);
    if (even && valid == ~0ull) {
      // one page per instruction: the addresses are scalar work
#pragma unroll
      for (int x = 0; x < NI; ++x) {
        const int first = 64 * (wave + NW * x), key = base + first / P;
        if ((uint32_t)(key - page_key) >= a.page.d) {
          const int pg = (int)fdiv(key, a.page);
          const int64_t page = pages.uniform_at(pg);
          page_key = pg * (int)a.page.d;
          kpage = kbase + page * a.k_page;
          vpage = vbase + page * a.v_page;
        }
        const int64_t off = (int64_t)(key - page_key) * ROW;
        dma16(kpage + off, koff, lds_addr(&smem_k[stage][first]));
        dma16(vpage + off, voff, lds_addr(&smem_v[stage][first]));
      }
      return valid;
    }
#pragma unroll 1
    for (int x = 0; x < NI; ++x) {
      const int first = 64 * (wave + NW * x);
      const int slot = first + lane, row = slot / P;
      const int pg = (int)fdiv(base + row, a.page), off = base + row - pg * (int)a.page.d;
      const int64_t page = pages.at(pg);
      const char* kp = kbase + page * a.k_page + (int64_t)(off - lane / P) * ROW + koff;
      const char* vp = vbase + page * a.v_page + (int64_t)(off - lane / P) * ROW + voff;
      if (!((valid >> row) & 1)) kp = vp = (const char*)&attn_zero;
      dma16(kp, lds_addr(&smem_k[stage][first]));
      dma16(vp, lds_addr(&smem_v[stage][first]));
    }
    return valid;
  };

  // A cache in 8 bits: each thread fetches NX pieces of 16 codes of a tile and their scales into
  // registers, half of them K's and then the same rows of V (or, where there is one, waves
  // of the first half K's and the others V's), and a step later widens them into a tile
  // that the matrix instructions read.
  constexpr int PC = DIM / 16, NX = Q8 ? 2 * PC / NW : 1, NR = NX > 1 ? NX / 2 : 1;
  u32x4v_t codes[NX];
  float scale[NX];
  const int wrow = (NX > 1 ? wave : wave % (NW / 2)) * (64 / PC);  // the wave's first row; others 64 NW / PC on
  auto of_v = [&](int x) __attribute__((always_inline)) { return NX > 1 ? x >= NR : wave >= NW / 2; };
  // Addresses are integers: a generic pointer would make every LDS read wait for the loads.
  auto get = [&](int x, uint64_t cp, uint64_t sp) __attribute__((always_inline)) {
    codes[x] = *(const __attribute__((address_space(1))) u32x4v_t*)cp;
    scale[x] = *(const __attribute__((address_space(1))) float*)sp;
  };
  const int64_t scale_page = [&] {
    if constexpr (Q8) return (int64_t)a.hkv * a.scales.per_page * 4;
    else return (int64_t)0;
  }();
  auto pool_of = [&](bool v) __attribute__((always_inline)) { return (uint64_t)(v ? vbase : kbase); };
  auto scales_of = [&](bool v) __attribute__((always_inline)) -> uint64_t {
    if constexpr (Q8) return (uint64_t)((v ? a.scales.v : a.scales.k) + (int64_t)kvh * a.scales.per_page);
    else return 0;
  };
  // Piece x where a load's rows share a page and every key is there: scalar work but for the scales.
  // V's use what the same rows of K have worked out.  For another tile it loads something that the
  // page or page 0 holds (16 bytes of a row, where rows of a load may lie on two), with no branch.
  const bool pages_fit = a.page.d % (64 / PC) == 0;
  const uint32_t fetch_byte = pages_fit ? 16 * lane : 0, fetch_row = pages_fit ? lane / PC : 0;
  uint32_t fpage[NR], fscale[NR];
  int foff[NR];
  auto fetch_whole = [&](int base, int x) __attribute__((always_inline)) {
    if constexpr (Q8) {
      const int r = x % NR;
      const bool v = of_v(x);
      if (x < NR) {
        const int key = base + wrow + r * (64 * NW / PC), pg = (int)fdiv(key, a.page);
        foff[r] = key - pg * (int)a.page.d;
        fpage[r] = (uint32_t)max(pages.uniform_at(pg), 0);
        fscale[r] = 4 * fdiv(foff[r] + fetch_row, a.scales.block);
      }
      // (a uniform address and an offset of 32 bits: no registers for sums of the two)
      typedef const __attribute__((address_space(1))) char* bytes_t;
      const bytes_t cp = (bytes_t)(pool_of(v) + fpage[r] * (uint64_t)(v ? a.v_page : a.k_page) +
                                   (uint64_t)foff[r] * DIM);
      const bytes_t sp = (bytes_t)(scales_of(v) + fpage[r] * (uint64_t)scale_page);
      codes[x] = *(const __attribute__((address_space(1))) u32x4v_t*)(cp + fetch_byte);
      scale[x] = *(const __attribute__((address_space(1))) float*)(sp + fscale[r]);
    }
  };
  auto fetch = [&](int base, uint64_t valid, int x) __attribute__((always_inline)) {  // any tile
    if constexpr (Q8) {
      const int ln = again(lane);  // or addresses would be kept for every x
      const int row = wrow + x % NR * (64 * NW / PC) + ln / PC, key = base + row;
      const int pg = (int)fdiv(key, a.page), off = key - pg * (int)a.page.d;
      const int64_t page = pages.at(pg);
      const bool v = of_v(x), is = (valid >> row) & 1;
      get(x, is ? pool_of(v) + page * (v ? a.v_page : a.k_page) + (int64_t)off * DIM + 16 * (ln % PC)
                : (uint64_t)&attn_zero,
          is ? scales_of(v) + page * scale_page + 4 * fdiv(off, a.scales.block) : (uint64_t)&attn_zero);
    }
  };
  // Where the first half of this lane's piece goes in stage 0; the second goes beside it.  (Eight lanes
  // write at a time, and take every other 16 bytes of 256: half of the banks.  Halves in turn would
  // take all of them, but the selects cost more than the conflicts: 4.15 ms against 4.05.)
  const int crow = wrow + lane / PC;
  const uint32_t kput = lds_addr(&smem_k[0][crow * P + (2 * (lane % PC) ^ kswz<P>(crow))]);
  const uint32_t vput = lds_addr(&smem_v[0][crow * P + (2 * (lane % PC) ^ vswz<P>(crow))]);
  static_assert(!Q8 || NR == 1 || 64 * NW / PC % 16 == 0, "a thread's rows agree modulo 16");
  auto widen = [&](int at, int x, int y) __attribute__((always_inline)) {  // half y; at: bytes of the stage
    if constexpr (Q8) {
      const bool v = of_v(x);
      if constexpr (CODE == INT8) {
        if (y == 0) {
          // Behind the step's product and reads, or the mask moves up to the fetch or before them and they
          // wait for the scale too (2048 tokens on 131072 keys: 4.22 ms, so 4.14, without a mask 4.10).
          __builtin_amdgcn_sched_barrier(0);
          asm volatile("" : "+v"(scale[x]));
          scale[x] = pow2_scale(scale[x]);
        }
      }
      const u32x2v_t lo = Code<CODE>::widen16(E{}, codes[x][2 * y], scale[x]);
      const u32x2v_t hi = Code<CODE>::widen16(E{}, codes[x][2 * y + 1], scale[x]);
      const uint32_t to = ((v ? vput : kput) ^ 16 * y) + at + x % NR * (64 * NW / PC) * ROW;
      *(__attribute__((address_space(3))) u32x4v_t*)(uintptr_t)to = u32x4v_t{lo[0], lo[1], hi[0], hi[1]};
    }
  };
  auto widen_all = [&](int at) __attribute__((always_inline)) {
#pragma unroll
    for (int x = 0; x < NX; ++x) {
      widen(at, x, 0);
      widen(at, x, 1);
    }
  };

  f32x16_t s[2];
  frag p[4];

  auto clear_scores = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int x = 0; x < 16; ++x) s[k][x] = 0.0f;
  };
  auto score = [&](int stage, int n) __attribute__((always_inline)) {  // S^T += K Q^T, step n
    const int x = n / 2, k = n % 2;
    s[k] = Half<E>::mma32(
        __builtin_bit_cast(frag, lds_read16(ka[x] + stage * STAGE + 32 * k * ROW)), q[x], s[k]);
  };
  auto value = [&](int stage, int n) __attribute__((always_inline)) {  // O^T += V^T P^T, step n
    const int kc = n / DV, d = n % DV;
    const uint32_t at = va[d] + stage * STAGE + 16 * kc * ROW;
    typedef short s16x8_t __attribute__((ext_vector_type(8)));
    const s16x4_t u = lds_read_tr(at), w = lds_read_tr(at + 8 * ROW);
    const s16x8_t z = {u[0], u[1], u[2], u[3], w[0], w[1], w[2], w[3]};
    o[d] = Half<E>::mma32(__builtin_bit_cast(frag, z), p[kc], o[d]);
  };
  // The products of a slot.  The scheduler is told to keep AHEAD fragments' reads in
  // flight: left to itself it waits for each one right before its product.
  constexpr int AHEAD = 3, NS = 2 * QS, NV = 4 * DV;
  // Over codes the order is spelled out (beside codes on their way the scheduler gives it up), with
  // other work between the products: `fill` of a step.
  auto nothing = [](int) {};
  auto scores = [&](int stage, auto fill) __attribute__((always_inline)) {
    clear_scores();
    if constexpr (Q8) {
      u32x4v_t f[AHEAD];
#pragma unroll
      for (int n = 0; n < NS + AHEAD; ++n) {
        if (n >= AHEAD) {
          const int x = (n - AHEAD) / 2, k = (n - AHEAD) % 2;
          s[k] = Half<E>::mma32(__builtin_bit_cast(frag, f[n % AHEAD]), q[x], s[k]);
        }
        if (n < NS) f[n % AHEAD] = lds_read16(ka[n / 2] + stage * STAGE + 32 * (n % 2) * ROW);
        fill(n);
        __builtin_amdgcn_sched_barrier(0);
      }
      return;
    }
#pragma unroll
    for (int n = 0; n < NS; ++n) score(stage, n);
    __builtin_amdgcn_sched_group_barrier(DS_READ, AHEAD, 0);
#pragma unroll
    for (int n = 0; n < NS - AHEAD; ++n) {
      __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
      __builtin_amdgcn_sched_group_barrier(DS_READ, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(MFMA, AHEAD, 0);
  };
  auto values = [&](int stage, auto fill) __attribute__((always_inline)) {
    if constexpr (Q8) {
      s16x4_t u[AHEAD], w[AHEAD];
#pragma unroll
      for (int n = 0; n < NV + AHEAD; ++n) {
        if (n >= AHEAD) {
          const int m = n % AHEAD, kc = (n - AHEAD) / DV, d = (n - AHEAD) % DV;
          typedef short s16x8_t __attribute__((ext_vector_type(8)));
          const s16x8_t z = {u[m][0], u[m][1], u[m][2], u[m][3], w[m][0], w[m][1], w[m][2], w[m][3]};
          o[d] = Half<E>::mma32(__builtin_bit_cast(frag, z), p[kc], o[d]);
        }
        if (n < NV) {
          const uint32_t at = va[n % DV] + stage * STAGE + 16 * (n / DV) * ROW;
          u[n % AHEAD] = lds_read_tr(at);
          w[n % AHEAD] = lds_read_tr(at + 8 * ROW);
        }
        fill(n);
        __builtin_amdgcn_sched_barrier(0);
      }
      return;
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) value(stage, n);
    __builtin_amdgcn_sched_group_barrier(DS_READ, 2 * AHEAD, 0);
#pragma unroll
    for (int n = 0; n < NV - AHEAD; ++n) {
      __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
      __builtin_amdgcn_sched_group_barrier(DS_READ, 2, 0);
    }
    __builtin_amdgcn_sched_group_barrier(MFMA, AHEAD, 0);
  };
  // Takes out the keys that are hidden from the row, or absent.
  auto hide = [&](int base, uint64_t valid) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t see = seen(a, base + 32 * k, qpos, (uint32_t)(valid >> (32 * k))) >> (4 * h);
#pragma unroll
      for (int x = 0; x < 16; ++x)
        s[k][x] = see & (1u << (8 * (x / 4) + x % 4)) ? s[k][x] : NEG_INF;
    }
  };
  auto softmax = [&]() __attribute__((always_inline)) {  // m, l, O rescaled; P
    float mx = NEG_INF;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int x = 0; x < 16; ++x) mx = fmaxf(mx, s[k][x]);
    mx = max_half(mx) * c;  // c > 0
    if (__any(mx > m + LAG)) {
      const float nm = fmaxf(m, mx);
      const float f = nm == NEG_INF ? 1.0f : exp2_fast(m - nm);
      m = nm;
      l *= f;
#pragma unroll
      for (int d = 0; d < DV; ++d)
#pragma unroll
        for (int x = 0; x < 16; ++x) o[d][x] *= f;
    }
    // a row that has seen no key yet keeps m = -inf: its scores are all -inf too
    const float mb = (m == NEG_INF ? 0.0f : m) - Half<E>::P_BIAS;
    // P^T as it lies: chunk kc of 16 keys, slots 0..3 keys 4 h + x, slots 4..7 keys 8 + 4 h + x
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const float e = exp2_fast(fmaf(s[k][x], c, -mb));
        l += e;
        Half<E>::set(p[2 * k + x / 8], x % 8, e);
      }
  };
  // The same on the vector unit, key by key, added where the key is visible: V may
  // hold infinities or NaN that some rows must not see (0 times them is NaN).
  auto values_by_key = [&](int base, int stage, uint64_t valid) __attribute__((always_inline)) {
    const uint4* const vt = smem_v[stage];
#pragma unroll 1
    for (int j = 0; j < KT; ++j) {
      // p of key j lies in slot e of chunk j / 16, in half (j / 4) % 2 of the wave
      const int e = (j & 3) | ((j >> 1) & 4);
      uint32_t w = 0;
#pragma unroll
      for (int x = 0; x < 16; ++x)
        w = 4 * (j >> 4) + (e >> 1) == x ? __builtin_bit_cast(u32x4v_t, p[x / 4])[x % 4] : w;
      const float pj =
          Half<E>::widen(__shfl(e & 1 ? w >> 16 : w & 0xffffu, l32 + 32 * ((j >> 2) & 1)));
      // all ones where this row sees the key
      const uint32_t see =
          0u - ((seen(a, base + (j & 32), qpos, (uint32_t)(valid >> (j & 32))) >> (j & 31)) & 1);
#pragma unroll
      for (int d = 0; d < DV; ++d) {
        __builtin_amdgcn_sched_barrier(0);  // few registers at a time
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint2 u = *reinterpret_cast<const uint2*>(
              reinterpret_cast<const char*>(vt + j * P + ((4 * d + x) ^ vswz<P>(j))) + 8 * h);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t v = (y < 2 ? u.x : u.y) & see;
            o[d][4 * x + y] = fmaf(pj, Half<E>::widen(y & 1 ? v >> 16 : v & 0xffffu), o[d][4 * x + y]);
          }
        }
      }
    }
  };

  auto clear = [&]() __attribute__((always_inline)) {
    m = NEG_INF;
    l = 0.0f;
#pragma unroll
    for (int d = 0; d < DV; ++d)
#pragma unroll
      for (int x = 0; x < 16; ++x) o[d][x] = 0.0f;
  };
  // Whether all of the wave's rows see all of the tile: those that start in
  // [whole_lo, whole_hi], or before the sinks end.
  const int whole_hi = wa - (KT - 1), whole_lo = a.window > 0 ? wb - a.window + 1 : 0;
  const int whole_sinks = a.sinks - KT;
  auto whole = [&](int base, uint64_t valid) __attribute__((always_inline)) {
    return base <= whole_hi && valid == ~0ull && (base >= whole_lo || base <= whole_sinks);
  };

  // The fragment addresses move between the halves of the ring, so that within one
  // every read's place is a constant.
  auto turn = [&](int by) __attribute__((always_inline)) {
#pragma unroll
    for (int x = 0; x < QS; ++x) ka[x] += by;
#pragma unroll
    for (int d = 0; d < DV; ++d) va[d] += by;
  };
  // The queries come through the half of the ring that the first tiles leave free,
  // 32 rows to a wave, laid out as K rows are: whole rows at a time, where fragments
  // straight from memory touch each row in eight pieces (24 ragged prompts of 33515
  // tokens: 822 us against 849 us).
  auto ask_queries = [&]() __attribute__((always_inline)) {
    uint4* const mine = wave < NW / 2 ? &smem_k[PAIR][wave * 32 * P] : &smem_v[PAIR][(wave - NW / 2) * 32 * P];
#pragma unroll
    for (int x = 0; x < P / 2; ++x) {
      const int row = (64 * x + lane) / P;
      const int lo = __builtin_amdgcn_ds_bpermute(4 * row, (int)qrow);
      const int hi = __builtin_amdgcn_ds_bpermute(4 * row, (int)(qrow >> 32));
      const int64_t at = ((int64_t)hi << 32) | (uint32_t)lo;
      const char* g = (const char*)a.q + 2 * at + 16 * (lane % P ^ kswz<P>(row));
      if (hi < 0) g = (const char*)&attn_zero;
      dma16(g, lds_addr(mine + 64 * x));
    }
    return mine;
  };
  auto take_queries = [&](const uint4* mine) __attribute__((always_inline)) {
    dma_wait<0>();
#pragma unroll
    for (int x = 0; x < QS; ++x)
      q[x] = __builtin_bit_cast(frag, lds_read16(ka[x] + lds_addr(mine) - lds_addr(&smem_k[0][0])));
  };
  // PAIR tiles between barriers, while the DMA fills the other half of the ring.  A
  // wave without rows (in a request's last tile) does its part of the loads only.
  auto walk = [&](auto busy) __attribute__((always_inline)) {
    constexpr bool BUSY = decltype(busy)::value;
    clear();
    uint64_t valid[PAIR], next[PAIR];  // the keys of the tiles
    int base[PAIR], nbase[PAIR];       // and where they start
    auto load = [&](int i, int half) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < PAIR; ++j) {
        next[j] = 0;
        nbase[j] = range.base(i + j);
        if (i + j < t1) next[j] = issue(nbase[j], half * PAIR + j);
      }
    };
    uint4* const mine = ask_queries();
    load(t0, 0);
    take_queries(mine);
    int half = 0;
#pragma unroll 1
    for (int i = t0; i < t1; i += PAIR, half ^= 1) {
#pragma unroll
      for (int j = 0; j < PAIR; ++j) {
        valid[j] = next[j];
        base[j] = nbase[j];
      }
      // these tiles have landed for every wave, and every wave is done with the last
      tile_barrier<0>();
      load(i + PAIR, half ^ 1);
      if constexpr (!BUSY) continue;
#pragma unroll
      for (int j = 0; j < PAIR; ++j) {
        if (i + j >= t1) break;
        __builtin_amdgcn_s_setprio(1);
        scores(j, nothing);
        __builtin_amdgcn_s_setprio(0);
        if (!whole(base[j], valid[j])) hide(base[j], valid[j]);
        softmax();
        __builtin_amdgcn_s_setprio(1);
        values(j, nothing);
        __builtin_amdgcn_s_setprio(0);
      }
      turn(half ? -PAIR * STAGE : PAIR * STAGE);
    }
    if (BUSY && half) turn(-PAIR * STAGE);
  };
  // The same over codes.  Tile t's step widens the codes of tile t + PAIR (fetched during the step
  // before) among its scores, into the half of the ring that the barrier has set free, and
  // fetches those of the tile after that among its values.
  auto walk_codes = [&](auto busy) __attribute__((always_inline)) {
    constexpr bool BUSY = decltype(busy)::value;
    constexpr int LOOK = PAIR + 1;
    clear();
    uint64_t valid[LOOK + 1];  // the keys of tiles t .. t + LOOK
    int base[LOOK + 1];        // and where they start
    auto find = [&](int t, int k) __attribute__((always_inline)) {
      base[k] = range.base(t);
      valid[k] = locate(base[k]);
    };
    auto fetch_any = [&](int k) __attribute__((always_inline)) {
#pragma unroll
      for (int x = 0; x < NX; ++x) fetch(base[k], valid[k], x);
    };
    const uint4* const mine = ask_queries();
#pragma unroll
    for (int x = 0; x < NX; ++x) {
      codes[x] = u32x4v_t{0, 0, 0, 0};
      scale[x] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < LOOK; ++j) {
      base[j] = 0;
      valid[j] = 0;
      if (t0 + j < t1) {
        find(t0 + j, j);
        fetch_any(j);
        if (j < PAIR) widen_all(j * STAGE);
      }
    }
    take_queries(mine);
    int half = 0;
#pragma unroll 1
    for (int i = t0; i < t1; i += PAIR, half ^= 1) {
      // these tiles are there for every wave, and every wave is done with the last
      lds_wait();
      __builtin_amdgcn_s_barrier();
      asm volatile("" : : : "memory");
      const int there = (half ^ 1) * (PAIR * STAGE);
#pragma unroll
      for (int j = 0; j < PAIR; ++j) {
        const int t = i + j;
        if (t >= t1) break;
        if constexpr (BUSY) {
          __builtin_amdgcn_s_setprio(1);
          scores(j, [&](int n) __attribute__((always_inline)) {
            const int m = n - AHEAD - 2;
            if (m >= 0 && m < 2 * NX) widen(there + j * STAGE, m / 2, m % 2);
          });
          __builtin_amdgcn_s_setprio(0);
          if (!whole(base[0], valid[0])) hide(base[0], valid[0]);
          softmax();
        } else {
          widen_all(there + j * STAGE);
        }
        valid[LOOK] = 0;
        base[LOOK] = 0;
        const bool more = t + LOOK < t1;
        if (more) find(t + LOOK, LOOK);
        if constexpr (BUSY) {
          __builtin_amdgcn_s_setprio(1);
          values(j, [&](int n) __attribute__((always_inline)) {
            if (n % 2 == 0 && n / 2 < NX) fetch_whole(base[LOOK], n / 2);
          });
          __builtin_amdgcn_s_setprio(0);
        } else {
#pragma unroll
          for (int x = 0; x < NX; ++x) fetch_whole(base[LOOK], x);
        }
        if (more && !(pages_fit && valid[LOOK] == ~0ull)) fetch_any(LOOK);
#pragma unroll
        for (int k = 0; k < LOOK; ++k) {
          valid[k] = valid[k + 1];
          base[k] = base[k + 1];
        }
      }
      if constexpr (BUSY) turn(half ? -PAIR * STAGE : PAIR * STAGE);
    }
    if (BUSY && half) turn(-PAIR * STAGE);
  };
  // The same tile by tile, with the hidden keys' values kept out of the sums.
  auto walk_carefully = [&]() __attribute__((always_inline)) {
    clear();
    if constexpr (Q8) {  // the queries anew, rather than kept through everything before
      const Place z = place(again(lane));
      const u32x4v_t* src = reinterpret_cast<const u32x4v_t*>(
          (const E*)a.q + (z.in ? (int64_t)(rt.start + z.tok) * a.q_stride + z.head * DIM : 0));
#pragma unroll
      for (int x = 0; x < QS; ++x)
        q[x] = __builtin_bit_cast(frag, z.in ? src[2 * x + h] : u32x4v_t{0, 0, 0, 0});
    }
#pragma unroll 1
    for (int i = t0; i < t1; ++i) {
      __syncthreads();
      const int base = range.base(i);
      uint64_t valid;
      if constexpr (Q8) {
        valid = locate(base);
#pragma unroll
        for (int x = 0; x < NX; ++x) {
          fetch(base, valid, x);
          widen(0, x, 0);
          widen(0, x, 1);
          __builtin_amdgcn_sched_barrier(0);  // few registers at a time
        }
      } else {
        valid = issue(base, 0);
      }
      dma_wait<0>();
      __syncthreads();
      scores(0, nothing);
      hide(base, valid);
      softmax();
      if (whole(base, valid)) values(0, nothing);
      else values_by_key(base, 0, valid);
    }
  };
  if constexpr (Q8) {
    if (32 * wave < rows) walk_codes(std::true_type{});
    else walk_codes(std::false_type{});
  } else {
    if (32 * wave < rows) walk(std::true_type{});
    else walk(std::false_type{});
  }
  // a hidden infinity or NaN of V has spoilt the sums of its tile: once more, carefully
  float z = 0.0f;  // becomes NaN if any sum is not finite
#pragma unroll
  for (int d = 0; d < DV; ++d)
#pragma unroll
    for (int x = 0; x < 16; ++x) z = fmaf(o[d][x], 0.0f, z);
  if (__syncthreads_or(z != 0.0f)) walk_carefully();

  int out_tok = tok, out_head = head;
  if constexpr (Q8) {
    const Place z = place(again(lane));
    out_tok = z.tok;
    out_head = z.head;
    if (!z.in) return;
  } else {
    if (!in) return;
  }
  l = sum_half(l);
  // a row that sees no key has l = 0: zeros, and a log-sum-exp of -inf
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const float lse2 = l == 0.0f ? NEG_INF : m - Half<E>::P_BIAS + __log2f(l);
  const int64_t row = (int64_t)(rt.start + out_tok) * a.hq + out_head;
  if (a.part_n != nullptr && split == 0 && h == 0) a.part_n[row] = splits;
  if (splits == 1) {
    if (a.lse != nullptr && h == 0) a.lse[row] = lse2 * LN2;
  } else if (h == 0) {
    a.part_lse[(int64_t)split * a.total * a.hq + row] = lse2;
  }
#pragma unroll
  for (int d = 0; d < DV; ++d)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      float y[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) y[z] = l == 0.0f ? 0.0f : o[d][4 * x + z] * inv;
      const int col = 32 * d + 8 * x + 4 * h;
      if (splits == 1)
        store4((E*)a.out + row * DIM + col, y[0], y[1], y[2], y[3]);
      else
        store4(a.part_o + ((int64_t)split * a.total * a.hq + row) * DIM + col, y[0], y[1], y[2], y[3]);
    }
}

}  // namespace
}  // namespace kda
