// Paged attention of long chunks of new tokens (bf16, fp16).
//
// The same one-pass softmax as the rows kernel, with the work of a matrix product:
// a workgroup holds 32 rows per wave and all its waves walk the keys together, 64
// at a time, from K and V tiles in LDS that the next ones replace while they are
// used.  S^T = K Q^T and O^T = V^T P^T run on 32 x 32 x 16 matrix instructions;
// lane l holds row l % 32 of its wave, in S^T as in O^T, so a row's maximum and sum
// take one swap between the wave's halves.
#include "kda_attn.hpp"

namespace kda {
namespace {

constexpr int KT = 64;    // keys per tile
constexpr int RING = 4;   // tiles in LDS
constexpr int MFMA = 0x8, DS_READ = 0x100;  // instruction classes of sched_group_barrier

__device__ __forceinline__ int kswz(int r) { return r & 7; }
// The transposing read takes 32 bytes of rows r .. r + 3 at two neighbouring
// 32-byte columns per half wave: with this the eight fall into different banks.
template <int P> __device__ __forceinline__ int vswz(int r) {
  return P == 16 ? 2 * (2 * (r & 3) + ((r >> 2) & 1)) : 2 * ((r & 2) | ((r >> 2) & 1));
}

template <typename E, int DIM, int NW>
__global__ __launch_bounds__(64 * NW, 2) void tiles_kernel(const AttnLaunch a) {
  typedef typename Half<E>::frag frag;
  constexpr int P = DIM / 8;            // 16-byte pieces per row
  constexpr int NI = P / NW > 0 ? P / NW : 1;  // DMA instructions per wave and tile
  constexpr int QS = DIM / 16, DV = DIM / 32;
  static_assert(P % NW == 0, "a tile splits evenly over the waves");
  __shared__ uint4 smem[RING][2][KT * P];

  const int lane = threadIdx.x & 63, wave = wave_of();
  const int l32 = lane & 31, h = lane >> 5;
  // later tiles have more keys: they go first
  const int64_t work = (int64_t)gridDim.x - 1 - blockIdx.x;
  const int kvh = (int)(work % a.hkv), split = blockIdx.y;
  const RowTile rt = find_tile<32 * NW>(a, (int)(work / a.hkv), lane);
  if (rt.first >= rt.rows || rt.rows <= a.rows_limit) return;
  const int rows = min(32 * NW, rt.rows - rt.first);
  const int seq = max(a.seq[rt.req], 0);
  const int pos0 = seq - rt.len;
  const KeyRange<KT> range(a, pos0 + (int)fdiv(rt.first, a.gdiv),
                           pos0 + (int)fdiv(rt.first + rows - 1, a.gdiv), seq);
  int per;
  const int splits = split_of(range.tiles, a.tile_splits, a.tile_min_keys / KT, per);
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
  const bool busy = 32 * wave < rows;
  frag q[QS];
  {
    const uint4* src = reinterpret_cast<const uint4*>(
        (const E*)a.q + (in ? (int64_t)(rt.start + tok) * a.q_stride + head * DIM : 0));
#pragma unroll
    for (int s = 0; s < QS; ++s)
      q[s] = __builtin_bit_cast(frag, in ? src[2 * s + h] : make_uint4(0, 0, 0, 0));
    // they arrive here: a wait for them in the loop would wait for the DMA too
#pragma unroll
    for (int s = 0; s < QS; ++s) asm volatile("" : "+v"(q[s]));
  }

  // LDS byte addresses of the fragments in stage 0: key row l32 of a K tile, and the
  // rows and columns that this lane points the transposing reads at (both swizzles
  // depend on the row modulo 8 alone, so the other rows are constants away)
  uint32_t ka[QS], va[DV];
#pragma unroll
  for (int x = 0; x < QS; ++x) ka[x] = lds_addr(&smem[0][0][l32 * P + ((2 * x + h) ^ kswz(l32))]);
#pragma unroll
  for (int d = 0; d < DV; ++d) {
    const int i16 = lane & 15, row = 4 * h + (i16 >> 2);
    const int piece = 4 * d + 2 * ((lane >> 4) & 1) + ((i16 & 3) >> 1);
    va[d] = lds_addr(&smem[0][1][row * P + (piece ^ vswz<P>(row))]) + 8 * (i16 & 1);
  }
  constexpr int STAGE = 2 * KT * P * 16, ROW = P * 16;  // bytes

  f32x16_t o[DV];
  float m, l;
  const float c = a.scale * LOG2E;

  PageWindow pages(a, rt.req);
  const char* const kbase = (const char*)a.kc + (int64_t)kvh * a.page.d * (DIM * 2);
  const char* const vbase = (const char*)a.vc + (int64_t)kvh * a.page.d * (DIM * 2);

  // Issues the DMA of key tile i; returns which of its keys exist.
  auto issue = [&](int i, int stage) __attribute__((always_inline)) -> uint64_t {
    const int base = range.base(i);
    const int p0 = (int)fdiv(base, a.page);
    const int p1 = (int)fdiv(min(base + KT - 1, (int)a.key_capacity - 1), a.page);
    pages.cover(a, p0, p1, lane);
    // inside the range and with every page there (the common case), all keys exist
    uint64_t valid = ~0ull;
    if (base + KT > range.end || !(base >= range.lo || base + KT <= range.sink_end) ||
        pages.missing(p0, p1)) {
      const int key = base + lane;
      valid = __ballot(range.has(key) && pages.at((int)fdiv(key, a.page)) >= 0);
    }
#pragma unroll
    for (int x = 0; x < NI; ++x) {
      const int first = 64 * (wave + NW * x);
      const int slot = first + lane, row = slot / P, ps = slot % P;
      const int pg = (int)fdiv(base + row, a.page), off = base + row - pg * (int)a.page.d;
      const int page = pages.at(pg);
      const char* kp = kbase + (int64_t)page * a.k_page + off * (DIM * 2) + 16 * (ps ^ kswz(row));
      const char* vp = vbase + (int64_t)page * a.v_page + off * (DIM * 2) + 16 * (ps ^ vswz<P>(row));
      if (valid != ~0ull && !((valid >> row) & 1)) kp = vp = (const char*)&attn_zero;
      dma16(kp, lds_addr(&smem[stage][0][first]));
      dma16(vp, lds_addr(&smem[stage][1][first]));
    }
    return valid;
  };

  f32x16_t s[2];
  frag p[4];

  // S^T = K Q^T.  The scheduler is told to keep AHEAD fragment reads in flight: left
  // to itself it waits for each one right before its product.
  auto scores = [&](int stage) __attribute__((always_inline)) {
    constexpr int AHEAD = 6, N = 2 * QS;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int x = 0; x < 16; ++x) s[k][x] = 0.0f;
#pragma unroll
    for (int x = 0; x < QS; ++x)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        s[k] = Half<E>::mma32(
            __builtin_bit_cast(frag, lds_read16(ka[x] + stage * STAGE + 32 * k * ROW)), q[x], s[k]);
    __builtin_amdgcn_sched_group_barrier(DS_READ, AHEAD, 0);
#pragma unroll
    for (int x = 0; x < N - AHEAD; ++x) {
      __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
      __builtin_amdgcn_sched_group_barrier(DS_READ, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(MFMA, AHEAD, 0);
  };
  auto hide = [&](int base, uint64_t valid) __attribute__((always_inline)) {  // keys hidden from the row, or absent
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
  auto values = [&](int stage) __attribute__((always_inline)) {  // O^T += V^T P^T
    constexpr int AHEAD = 6, N = 4 * DV;
#pragma unroll
    for (int kc = 0; kc < 4; ++kc)
#pragma unroll
      for (int d = 0; d < DV; ++d) {
        const uint32_t at = va[d] + stage * STAGE + 16 * kc * ROW;
        typedef short s16x8_t __attribute__((ext_vector_type(8)));
        const s16x4_t u = lds_read_tr(at), w = lds_read_tr(at + 8 * ROW);
        const s16x8_t z = {u[0], u[1], u[2], u[3], w[0], w[1], w[2], w[3]};
        o[d] = Half<E>::mma32(__builtin_bit_cast(frag, z), p[kc], o[d]);
      }
    __builtin_amdgcn_sched_group_barrier(DS_READ, 2 * AHEAD, 0);
#pragma unroll
    for (int x = 0; x < N - AHEAD; ++x) {
      __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
      __builtin_amdgcn_sched_group_barrier(DS_READ, 2, 0);
    }
    __builtin_amdgcn_sched_group_barrier(MFMA, AHEAD, 0);
  };
  // The same on the vector unit, key by key, added where the key is visible: V may
  // hold infinities or NaN that some rows must not see (0 times them is NaN).
  auto values_by_key = [&](int base, int stage, uint64_t valid) __attribute__((always_inline)) {
    const uint4* const vt = smem[stage][1];
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
  // Whether any of the wave's rows sees a key of the tile, and whether all of them
  // see all of it.
  auto visible = [&](int base) __attribute__((always_inline)) {
    return busy && base <= wb && !(a.window > 0 && base + KT - 1 <= wa - a.window && base >= a.sinks);
  };
  auto whole = [&](int base, uint64_t valid) __attribute__((always_inline)) {
    return base + KT - 1 <= wa && valid == ~0ull &&
           !(a.window > 0 && base <= wb - a.window && base + KT > a.sinks);
  };

  // The two waves of a SIMD take turns: while one is at its matrix products (O of the
  // last tile, S of this one) the other is at its softmax, a barrier apart.  Slot
  // 2 i: waves 0 .. 3 multiply for tile i, the others take the softmax of tile i - 1;
  // slot 2 i + 1: the other way round.  Tile j is asked for in slots 2 j - 4 and
  // 2 j - 3, the last reader of tile j - 4 was in slot 2 j - 5, and it has landed by
  // slot 2 j.
  auto walk = [&]() __attribute__((always_inline)) {
    const bool late = wave >= NW / 2;
    const int nt = t1 - t0;
    clear();
    if (nt <= 0) return;
    uint64_t v0 = ~0ull, v1 = ~0ull, v2 = ~0ull;  // the keys of tiles i, i + 1, i + 2
#pragma unroll 1
    for (int i = 0; i < 2 && i < nt; ++i) {
      v0 = v1;
      v1 = issue(t0 + i, i);
    }
    if (nt == 1) v0 = v1;
    dma_wait<0>();
    __builtin_amdgcn_s_barrier();
    if (late) __builtin_amdgcn_s_barrier();
    bool live = false;  // P holds tile i - 1
#pragma unroll 1
    for (int i = 0; i < nt; ++i) {
      const int base = range.base(t0 + i);
      const bool vis = visible(base);
      if (i + 2 < nt) v2 = issue(t0 + i + 2, (i + 2) % RING);
      if (live) values((i + RING - 1) % RING);
      if (vis) scores(i % RING);
      lds_wait();
      if (late) {
        if (i + 2 < nt) dma_wait<2 * NI>();
        else dma_wait<0>();
      }
      __builtin_amdgcn_s_barrier();
      if (vis) {
        if (!whole(base, v0)) hide(base, v0);
        softmax();
      }
      live = vis;
      if (!late) {
        if (i + 2 < nt) dma_wait<2 * NI>();
        else dma_wait<0>();
      }
      v0 = v1;
      v1 = v2;
      __builtin_amdgcn_s_barrier();
    }
    if (live) values((nt - 1) % RING);
    if (!late) __builtin_amdgcn_s_barrier();
  };
  // The same tile by tile, with the hidden keys' values kept out of the sums.
  auto walk_carefully = [&]() __attribute__((always_inline)) {
    clear();
#pragma unroll 1
    for (int i = t0; i < t1; ++i) {
      __syncthreads();
      const int base = range.base(i);
      const uint64_t valid = issue(i, 0);
      dma_wait<0>();
      __syncthreads();
      if (!visible(base)) continue;
      scores(0);
      hide(base, valid);
      softmax();
      if (whole(base, valid)) values(0);
      else values_by_key(base, 0, valid);
    }
  };
  walk();
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
  hipLaunchKernelGGL((tiles_kernel<E, DIM, NW>), dim3((unsigned)(tiles * L.hkv), (unsigned)L.tile_splits),
                     dim3(64 * NW), 0, (hipStream_t)L.stream, L);
  return hipGetLastError();
}
template <typename E, int DIM> hipError_t tiles_nw(const AttnLaunch& L) {
  return tiles_go<E, DIM, 8>(L);
}
template <typename E> hipError_t tiles_dim(const AttnLaunch& L) {
  return L.dim == 64 ? tiles_nw<E, 64>(L) : tiles_nw<E, 128>(L);
}

}  // namespace

hipError_t launch_attn_tiles(const AttnLaunch& L) {
  return L.dtype == 1 ? tiles_dim<bf16>(L) : tiles_dim<_Float16>(L);
}

}  // namespace kda
