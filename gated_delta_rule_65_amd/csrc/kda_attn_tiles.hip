// Paged attention of long chunks of new tokens (bf16, fp16).
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
#include "kda_attn.hpp"

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

template <typename E, int DIM, int NW>
__global__ __launch_bounds__(64 * NW, 2) void tiles_kernel(const AttnLaunch a) {
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
  const char* const kbase = (const char*)a.kc + (int64_t)kvh * a.page.d * (DIM * 2);
  const char* const vbase = (const char*)a.vc + (int64_t)kvh * a.page.d * (DIM * 2);

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

  // Issues the DMA of the key tile at `base`; returns which of its keys exist.
  auto issue = [&](int base, int stage) __attribute__((always_inline)) -> uint64_t {
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
  auto scores = [&](int stage) __attribute__((always_inline)) {
    clear_scores();
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
  auto values = [&](int stage) __attribute__((always_inline)) {
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
    // The queries come through the half of the ring that the first tiles leave free,
    // 32 rows to a wave, laid out as K rows are: whole rows at a time, where fragments
    // straight from memory touch each row in eight pieces (24 ragged prompts of 33515
    // tokens: 822 us against 849 us).
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
    load(t0, 0);
    dma_wait<0>();
#pragma unroll
    for (int x = 0; x < QS; ++x)
      q[x] = __builtin_bit_cast(frag, lds_read16(ka[x] + lds_addr(mine) - lds_addr(&smem_k[0][0])));
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
        scores(j);
        __builtin_amdgcn_s_setprio(0);
        if (!whole(base[j], valid[j])) hide(base[j], valid[j]);
        softmax();
        __builtin_amdgcn_s_setprio(1);
        values(j);
        __builtin_amdgcn_s_setprio(0);
      }
      turn(half ? -PAIR * STAGE : PAIR * STAGE);
    }
    if (BUSY && half) turn(-PAIR * STAGE);
  };
  // The same tile by tile, with the hidden keys' values kept out of the sums.
  auto walk_carefully = [&]() __attribute__((always_inline)) {
    clear();
#pragma unroll 1
    for (int i = t0; i < t1; ++i) {
      __syncthreads();
      const int base = range.base(i);
      const uint64_t valid = issue(base, 0);
      dma_wait<0>();
      __syncthreads();
      scores(0);
      hide(base, valid);
      softmax();
      if (whole(base, valid)) values(0);
      else values_by_key(base, 0, valid);
    }
  };
  if (32 * wave < rows) walk(std::true_type{});
  else walk(std::false_type{});
  // a hidden infinity or NaN of V has spoilt the sums of its tile: once more, carefully
  float z = 0.0f;  // becomes NaN if any sum is not finite
#pragma unroll
  for (int d = 0; d < DV; ++d)
#pragma unroll
    for (int x = 0; x < 16; ++x) z = fmaf(o[d][x], 0.0f, z);
  if (__syncthreads_or(z != 0.0f)) walk_carefully();

  if (!in) return;
  l = sum_half(l);
  // a row that sees no key has l = 0: zeros, and a log-sum-exp of -inf
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const float lse2 = l == 0.0f ? NEG_INF : m - Half<E>::P_BIAS + __log2f(l);
  const int64_t row = (int64_t)(rt.start + tok) * a.hq + head;
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

template <typename E, int DIM, int NW> hipError_t tiles_go(const AttnLaunch& L) {
  const int64_t tiles = (int64_t)L.total * L.group / (32 * NW) + L.n;
  hipLaunchKernelGGL((tiles_kernel<E, DIM, NW>), dim3((unsigned)(tiles * L.hkv), (unsigned)L.splits),
                     dim3(64 * NW), 0, (hipStream_t)L.stream, L);
  return hipGetLastError();
}
template <typename E, int DIM> hipError_t tiles_nw(const AttnLaunch& L) {
  return L.tile_waves == 8 ? tiles_go<E, DIM, 8>(L) : tiles_go<E, DIM, 4>(L);
}
template <typename E> hipError_t tiles_dim(const AttnLaunch& L) {
  return L.dim == 64 ? tiles_nw<E, 64>(L) : tiles_nw<E, 128>(L);
}

}  // namespace

hipError_t launch_attn_tiles(const AttnLaunch& L) {
  return L.dtype == 1 ? tiles_dim<bf16>(L) : tiles_dim<_Float16>(L);
}

}  // namespace kda
