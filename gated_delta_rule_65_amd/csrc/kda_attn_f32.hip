// Paged attention of chunks of new tokens in fp32, at full precision.
//
// The one-pass softmax of the other kernels on 16 x 16 x 4 matrix instructions.  A
// workgroup of four waves holds 128 rows of one kv head, 32 to a wave, and all of them
// walk the keys together, 16 at a time, from one ring of K and V tiles in LDS: a tile
// crosses L2 once for the 128 rows.
//
// Bound by the matrix cores where chunks are long: a tile costs a wave 128 products (4096
// cycles for 128 channels), a SIMD holds two waves, and the ring keeps three tiles on
// their way.  2048 tokens on 8192 keys, 8 heads on 2, 128 channels: 540 to 560 us a call, 112
// to 107 TFLOP/s (507 to 514 of them this kernel, 23 the join), where a large library
// product reaches 154; with the keys split over the waves, each of which then reads every
// row tile's keys from L2 by itself, 690 us.  Products first and V reads three ahead of
// them brought 576 us to 560; two tiles a barrier change nothing.  Short chunks leave the
// matrix cores idle: 840 tokens take 34 us at 20 % (the rows kernel has those below 256
// rows).
#include "kda_attn.hpp"

namespace kda {
namespace {

constexpr int KT = 16, RB = 2, WAVES = 4;  // keys per tile, 16-row blocks per wave
constexpr int RING = 4, LOOK = RING - 1;   // tiles in LDS, tiles on their way
constexpr int AHEAD = 3;                   // V reads ahead of their products
constexpr int MFMA = 0x8, DS_READ = 0x100;  // instruction classes of sched_group_barrier

// Piece p of row r of a K tile sits in slot p ^ r of the row, so that a fragment read,
// one piece each of the 16 rows, spreads over the 256 bytes of all banks.  V is read 16
// floats of 4 rows at a time: rows 4 apart go to different 64 bytes.
__device__ __forceinline__ int vswz(int r) { return 4 * ((r >> 2) & 3); }

struct Tile {
  int base;        // its first key
  uint32_t valid;  // which of its keys exist
};

template <int DIM> __global__ __launch_bounds__(64 * WAVES, 2) void chunks_kernel(const AttnLaunch a) {
  constexpr uint32_t ALL = 0xffffu;
  constexpr int P = DIM / 4, QS = P / 4;        // 16-byte pieces per row; of a query, per lane
  constexpr int ROWS = 64 / P, ROW = 4 * DIM;   // keys of a DMA instruction, bytes of one
  constexpr int NI = KT / ROWS / WAVES;         // DMA instructions per wave and tile, K or V
  constexpr int STAGE = 2 * KT * P;             // pieces of a K and a V tile
  __shared__ __attribute__((aligned(1024))) uint4 smem[RING * STAGE];

  const int lane = threadIdx.x & 63, wave = wave_of();
  const int l16 = lane & 15, gq = lane >> 4;
  // later tiles have more keys: they go first
  const uint32_t work = gridDim.x - 1 - blockIdx.x, unit = fdiv(work, a.hdiv);
  const int kvh = (int)(work - unit * a.hkv), split = blockIdx.y;
  const RowTile rt = find_tile<CHUNK_ROWS>(a, (int)unit, lane);
  if (rt.first >= rt.rows || rt.rows == 0) return;
  const int rows = min(CHUNK_ROWS, rt.rows - rt.first);
  const int seq = rt.seq, pos0 = seq - rt.len;
  const KeyRange<KT> range(a, pos0 + (int)fdiv(rt.first, a.gdiv),
                           pos0 + (int)fdiv(rt.first + rows - 1, a.gdiv), seq);
  int per;
  const int splits = split_of(range.tiles, a.splits, a.min_keys / KT, per);
  if (split >= splits) return;
  const int t0 = split * per, t1 = min(range.tiles, t0 + per);

  // this lane's rows (the MFMA columns l16 of each block): their queries, zero past the
  // last row, and their positions
  const bool busy = 16 * RB * wave < rows;
  const float c = a.scale * LOG2E;
  u32x4v_t q[RB][QS];
  int qpos[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int r = 16 * (RB * wave + b) + l16;
    const int tok = (int)fdiv(rt.first + r, a.gdiv);
    const int head = kvh * a.group + rt.first + r - tok * a.group;
    qpos[b] = pos0 + tok;
    const bool in = r < rows;
    const u32x4v_t* src = reinterpret_cast<const u32x4v_t*>(
        (const float*)a.q + (in ? (int64_t)(rt.start + tok) * a.q_stride + head * DIM : 0));
#pragma unroll
    for (int s = 0; s < QS; ++s) q[b][s] = in ? src[4 * s + gq] : u32x4v_t{0, 0, 0, 0};
  }
  // positions of the wave's first and last row
  const int wa = pos0 + (int)fdiv(rt.first + 16 * RB * wave, a.gdiv);
  const int wb = pos0 + (int)fdiv(rt.first + min(16 * RB * (wave + 1), rows) - 1, a.gdiv);

  // This lane's piece of an instruction's keys, as bytes from the first of them; the
  // instruction's first row adds its own bits to the swizzles.
  const uint32_t koff = lane / P * ROW + 16 * (lane % P ^ lane / P);
  const uint32_t voff = lane / P * ROW + 16 * (lane % P);
  // LDS byte addresses of fragments in the first stage.  K: key l16, piece 4 i + gq; V: key
  // 4 gq + e, column 16 d + l16.  i and d change bits of their own.
  const uint32_t ka = lds_addr(smem + l16 * P + (gq ^ l16));
  const uint32_t va = lds_addr(smem + KT * P + 4 * gq * P + ((l16 >> 2) ^ vswz(4 * gq))) + 4 * (l16 & 3);
  const bool even = a.page.d % ROWS == 0;  // whether an instruction's keys share a page
  PageWindow pages(a, rt.req);
  const char* const kbase = (const char*)a.kc + (int64_t)kvh * a.page.d * ROW;
  const char* const vbase = (const char*)a.vc + (int64_t)kvh * a.page.d * ROW;

  // Issues this wave's part of the DMA of key tile i.
  auto issue = [&](int i, int stage) __attribute__((always_inline)) {
    Tile t;
    t.base = range.base(i);
    const int last = min(t.base + KT - 1, (int)a.key_capacity - 1);
    pages.cover(a, t.base, last, lane);
    // inside the range and with every page there (the common case), all keys exist
    t.valid = ALL;
    if (t.base + KT > range.end || !(t.base >= range.lo || t.base + KT <= range.sink_end) ||
        pages.missing(a, t.base, last)) {
      const int key = t.base + l16;
      const int page = pages.at((int)fdiv(key, a.page));  // of every lane's key
      t.valid = (uint32_t)__ballot(range.has(key) && page >= 0) & ALL;
    }
    uint4* const kt = smem + stage * STAGE;
    uint4* const vt = kt + KT * P;
#pragma unroll
    for (int x = 0; x < NI; ++x) {
      const int r0 = ROWS * (NI * wave + x);  // the instruction's first key
      if (even && t.valid == ALL) {
        // one page: the addresses are scalar work
        const int key = t.base + r0, pg = (int)fdiv(key, a.page);
        const int64_t off = key - pg * (int)a.page.d, page = pages.uniform_at(pg);
        dma16(kbase + page * a.k_page + off * ROW, koff ^ 16 * r0, lds_addr(kt + r0 * P));
        dma16(vbase + page * a.v_page + off * ROW, voff ^ 16 * vswz(r0), lds_addr(vt + r0 * P));
      } else {
        const int r = r0 + lane / P, key = t.base + r, pg = (int)fdiv(key, a.page);
        const int64_t off = key - pg * (int)a.page.d, page = pages.at(pg);
        const char* kp = kbase + page * a.k_page + off * ROW + 16 * (lane % P ^ r);
        const char* vp = vbase + page * a.v_page + off * ROW + 16 * (lane % P ^ vswz(r));
        if (!((t.valid >> r) & 1)) kp = vp = (const char*)&attn_zero;
        dma16(kp, lds_addr(kt + r0 * P));
        dma16(vp, lds_addr(vt + r0 * P));
      }
    }
    return t;
  };

  f32x4_t o[DIM / 16][RB], s[RB];
  float m[RB], l[RB];

  auto scores = [&](int stage) __attribute__((always_inline)) {  // S^T = K Q^T
    uint32_t at = ka + stage * (STAGE * 16);
    asm volatile("" : "+v"(at));  // or every step would keep its address
#pragma unroll
    for (int b = 0; b < RB; ++b) s[b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < QS; ++i) {
      const f32x4_t k = __builtin_bit_cast(f32x4_t, lds_read16(at ^ 64 * i));
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int b = 0; b < RB; ++b)
          s[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(k[e], __builtin_bit_cast(f32x4_t, q[b][i])[e],
                                                      s[b], 0, 0, 0);
    }
    __builtin_amdgcn_sched_group_barrier(DS_READ, 2, 0);
#pragma unroll
    for (int i = 0; i < QS - 2; ++i) {
      __builtin_amdgcn_sched_group_barrier(MFMA, 4 * RB, 0);
      __builtin_amdgcn_sched_group_barrier(DS_READ, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(MFMA, 8 * RB, 0);
  };
  // m, l, O rescaled; the probabilities take the scores' place.  `some` rows do not see
  // some of the keys.
  auto softmax = [&](const Tile& t, bool some) __attribute__((always_inline)) {
    if (some) {
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const uint32_t see = seen(a, t.base, qpos[b], t.valid) >> (4 * gq);
#pragma unroll
        for (int r = 0; r < 4; ++r) s[b][r] = see & (1u << r) ? s[b][r] : NEG_INF;
      }
    }
    float mx[RB];
    bool grew = false;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      float x = NEG_INF;
#pragma unroll
      for (int r = 0; r < 4; ++r) x = fmaxf(x, s[b][r]);
      mx[b] = max_quarter(x) * c;  // c > 0
      grew |= mx[b] > m[b] + LAG;
    }
    if (__any(grew)) {
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
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      // a row that has seen no key yet keeps m = -inf: its scores are all -inf too
      const float mb = m[b] == NEG_INF ? 0.0f : m[b];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[b][r] = exp2_fast(fmaf(s[b][r], c, -mb));
        l[b] += s[b][r];
      }
    }
  };
  auto values = [&](int stage) __attribute__((always_inline)) {  // O^T += V^T P^T
    uint32_t at = va + stage * (STAGE * 16);
    asm volatile("" : "+v"(at));
#pragma unroll
    for (int d = 0; d < DIM / 16; ++d) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = lds_read4((at ^ 64 * d) + e * ROW);
#pragma unroll
        for (int b = 0; b < RB; ++b)
          o[d][b] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, s[b][e], o[d][b], 0, 0, 0);
      }
    }
    // (the reads of two keys make one instruction)
    constexpr int NV = DIM / 8;
    __builtin_amdgcn_sched_group_barrier(DS_READ, AHEAD, 0);
#pragma unroll
    for (int n = 0; n < NV - AHEAD; ++n) {
      __builtin_amdgcn_sched_group_barrier(MFMA, 2 * RB, 0);
      __builtin_amdgcn_sched_group_barrier(DS_READ, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(MFMA, 2 * RB * AHEAD, 0);
  };
  // The same key by key on the vector unit, added where the key is visible: V may hold
  // infinities or NaN that some rows must not see (0 times them is NaN).
  auto values_by_key = [&](const Tile& t, int stage) __attribute__((always_inline)) {
    const uint4* const vt = smem + stage * STAGE + KT * P;
#pragma unroll 1
    for (int j = 0; j < KT; ++j) {
      float p[RB];
      uint32_t see[RB];  // all ones where the row sees the key
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        float x = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) x = (j & 3) == r ? s[b][r] : x;
        p[b] = __shfl(x, l16 + 16 * (j >> 2));
        see[b] = 0u - ((seen(a, t.base, qpos[b], t.valid) >> j) & 1);
      }
#pragma unroll
      for (int d = 0; d < DIM / 16; ++d) {
        __builtin_amdgcn_sched_barrier(0);
        const u32x4v_t v = __builtin_bit_cast(u32x4v_t, vt[j * P + ((4 * d + gq) ^ vswz(j))]);
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[d][b][i] = fmaf(p[b], __uint_as_float(v[i] & see[b]), o[d][b][i]);
      }
    }
  };

  auto walk = [&](auto careful) __attribute__((always_inline)) {
    constexpr bool CAREFUL = decltype(careful)::value;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      m[b] = NEG_INF;
      l[b] = 0.0f;
#pragma unroll
      for (int d = 0; d < DIM / 16; ++d) o[d][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    Tile ahead[LOOK];
#pragma unroll
    for (int j = 0; j < LOOK; ++j) {
      ahead[j] = Tile{0, 0};
      if (t0 + j < t1) ahead[j] = issue(t0 + j, j);
    }
    // the queries arrive here: a wait for them in the loop would wait for the DMA too
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int x = 0; x < QS; ++x) asm volatile("" : "+v"(q[b][x]));
    int stage = 0;
#pragma unroll 1
    for (int i = t0; i < t1; ++i, stage = (stage + 1) % RING) {
      const Tile t = ahead[0];
      // this tile has landed for every wave, and every wave is done with the one before
      if (i + LOOK - 1 < t1) tile_barrier<2 * NI * (LOOK - 1)>();
      else tile_barrier<0>();
#pragma unroll
      for (int j = 0; j + 1 < LOOK; ++j) ahead[j] = ahead[j + 1];
      if (i + LOOK < t1) ahead[LOOK - 1] = issue(i + LOOK, (stage + LOOK) % RING);
      if (!busy || t.base > wb) continue;  // none of the wave's rows sees it
      const bool some = t.valid != ALL || t.base + KT - 1 > wa ||
                        (a.window > 0 && t.base <= wb - a.window && t.base + KT > a.sinks);
      __builtin_amdgcn_s_setprio(1);
      scores(stage);
      __builtin_amdgcn_s_setprio(0);
      softmax(t, some);
      if constexpr (CAREFUL) {
        if (some) {
          values_by_key(t, stage);
          continue;
        }
      }
      __builtin_amdgcn_s_setprio(1);
      values(stage);
      __builtin_amdgcn_s_setprio(0);
    }
  };
  walk(std::false_type{});
  // a hidden infinity or NaN of V has spoilt the sums of its tile: once more, carefully
  float z = 0.0f;  // becomes NaN if any sum is not finite
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int d = 0; d < DIM / 16; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) z = fmaf(o[d][b][r], 0.0f, z);
  if (__syncthreads_or(z != 0.0f)) walk(std::true_type{});

#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const float sum = sum_quarter(l[b]);
    const int r = 16 * (RB * wave + b) + l16;
    if (r >= rows) continue;
    // a row that sees no key has sum 0: zeros, and a log-sum-exp of -inf
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const float lse2 = sum == 0.0f ? NEG_INF : m[b] + __log2f(sum);
    const int tok = (int)fdiv(rt.first + r, a.gdiv);
    const int head = kvh * a.group + rt.first + r - tok * a.group;
    const int64_t row = (int64_t)(rt.start + tok) * a.hq + head;
    const int64_t part = splits == 1 ? row : (int64_t)split * a.total * a.hq + row;
    if (gq == 0) {
      if (a.part_n != nullptr && split == 0) a.part_n[row] = splits;
      if (splits > 1) a.part_lse[part] = lse2;
      else if (a.lse != nullptr) a.lse[row] = lse2 * LN2;
    }
    float* const dst = (splits == 1 ? (float*)a.out : a.part_o) + part * DIM + 4 * gq;
#pragma unroll
    for (int d = 0; d < DIM / 16; ++d) {
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = sum == 0.0f ? 0.0f : o[d][b][i] * inv;
      store4(dst + 16 * d, y[0], y[1], y[2], y[3]);
    }
  }
}

template <int DIM> hipError_t chunks_go(const AttnLaunch& L) {
  const int64_t tiles = (int64_t)L.total * L.group / CHUNK_ROWS + L.n;
  hipLaunchKernelGGL((chunks_kernel<DIM>), dim3((unsigned)(tiles * L.hkv), (unsigned)L.splits),
                     dim3(64 * WAVES), 0, (hipStream_t)L.stream, L);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_chunks(const AttnLaunch& L) {
  return L.dim == 64 ? chunks_go<64>(L) : chunks_go<128>(L);
}

}  // namespace kda
