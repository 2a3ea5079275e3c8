// Paged attention of few rows per request (decode, short drafts; in fp32 also short
// chunks), and the join of split partials.
//
// out = softmax(scale q K^T) V over a request's visible keys, in one pass with
// the running maximum m and sum l of the softmax (exponents in base 2, the scale
// folded into them).  A workgroup of four waves holds 16 or 32 rows of one kv
// head; each wave walks its own quarter of the keys, so no barrier stands in the
// loop, and the four (m, l, O) are joined through LDS at the end.
//
// Bound by HBM: a key's K and V rows (512 bytes for 128 bf16 channels) are read
// once for all rows of the tile.  Each wave keeps a whole tile of 16 keys in flight
// by DMA into its own LDS double buffer while it works on the one before; with 64 KB
// a workgroup, two of them share a compute unit, and one streams while the other
// starts or joins.  256 ragged decode requests (1.7 GB of keys and values): 310 us, 5.5
// TB/s, where a plain read reaches 6.3; with tiles of 32 keys and one workgroup per
// unit it was 440 us, and a third buffer, a single one, or shorter splits change
// nothing.  In fp32 (3.4 GB) 620 to 660 us, with 4 tokens a request in bf16 324 to 332 us.
#include "kda_attn.hpp"

namespace kda {
namespace {

constexpr int WAVES = 4;

// Piece p of row r of a K tile sits in slot p ^ kswz(r) of the row: a fragment read
// takes one piece each of the 16 rows, which spread over the 256 bytes of all banks.
template <int P> __device__ __forceinline__ int kswz(int r) { return P >= 16 ? r : r >> 1; }
// V tiles are read 4 (16-bit) or 1 (fp32) columns by row groups: the slots of
// rows that one read touches together fall into different 32- (64-) byte columns.
template <typename E, int P> __device__ __forceinline__ int vswz(int r) {
  if (sizeof(E) == 4) return 4 * ((r >> 2) & 3);
  return P == 16 ? 2 * (r & 7) : 2 * ((r >> 1) & 3);
}

template <typename E, int DIM, int RB> struct Rows {
  static constexpr bool F32 = sizeof(E) == 4;
  static constexpr int KT = 16;                         // keys per tile
  static constexpr int P = DIM * (int)sizeof(E) / 16;  // 16-byte pieces per row
  static constexpr int NI = KT * P / 64;               // DMA instructions per K or V tile
  static constexpr int QS = P / 4;                     // Q pieces per lane and row block
  static constexpr int STAGE = 2 * KT * P;             // pieces of a K and a V tile
  // fp32 products take longer than a tile's way from memory: one buffer each for K and
  // V, refilled as soon as it is read, leaves room for a second workgroup
  static constexpr int STAGES = F32 ? 1 : 2;
  static constexpr int OS = DIM + 4;                   // floats per joined row (padded)
  static constexpr int JOIN = WAVES * 16 * RB * OS / 4;
  static constexpr int PIECES = WAVES * STAGES * STAGE > JOIN ? WAVES * STAGES * STAGE : JOIN;
};

// One key tile on its way: where it starts and which of its keys exist.
struct Tile {
  int base;
  uint32_t valid;
};

template <typename E, int DIM, int RB, bool BY_REQUEST>
__global__ __launch_bounds__(256, 2) void rows_kernel(const AttnLaunch a) {
  using R = Rows<E, DIM, RB>;
  constexpr uint32_t ALL = 0xffffu;
  constexpr int KT = R::KT, P = R::P, NI = R::NI, QS = R::QS;
  __shared__ __attribute__((aligned(1024))) uint4 smem[R::PIECES];
  __shared__ float sm_m[WAVES][16 * RB], sm_l[WAVES][16 * RB];

  const int lane = threadIdx.x & 63, wave = wave_of();
  const int l16 = lane & 15, gq = lane >> 4;
  // heads fastest, so that neighbouring workgroups (and one XCD's) share pages
  const uint32_t unit = fdiv(blockIdx.x, a.hdiv);
  const int kvh = (int)(blockIdx.x - unit * a.hkv), split = blockIdx.y;
  const RowTile rt = BY_REQUEST ? request_tile(a, (int)unit) : find_tile<16 * RB>(a, (int)unit, lane);
  if (rt.rows == 0) return;
  const int seq = rt.seq, pos0 = seq - rt.len;
  const float c = a.scale * LOG2E;
  constexpr float BIAS = [] {
    if constexpr (R::F32) return 0.0f;
    else return Half<E>::P_BIAS;
  }();
  uint4* const my = smem + wave * R::STAGES * R::STAGE;
  constexpr int ROWS = 64 / P, ROW = DIM * (int)sizeof(E);  // keys of a DMA instruction, bytes of one
  // this lane's piece of an instruction's keys, as bytes from the first of them
  const uint32_t koff = lane / P * ROW + 16 * (lane % P ^ kswz<P>(lane / P));
  const uint32_t voff = lane / P * ROW + 16 * (lane % P ^ vswz<E, P>(lane / P));
  // LDS byte addresses of fragments in the first stage.  K: key l16, piece 4 i + gq.
  // V, fp32: key 4 gq + e, column 16 d + l16; 16-bit, for the transposing read: columns
  // 16 d + 4 (l16 % 4) .. of key 4 gq + l16 / 4.  i and d change bits of their own.
  const uint32_t ka = lds_addr(my + l16 * P + (gq ^ kswz<P>(l16)));
  const int vrow = R::F32 ? 4 * gq : 4 * gq + (l16 >> 2);
  const int vpiece = R::F32 ? l16 >> 2 : (l16 & 3) >> 1;
  const uint32_t va = lds_addr(my + KT * P + vrow * P + (vpiece ^ vswz<E, P>(vrow))) +
                      (R::F32 ? 4 * (l16 & 3) : 8 * (l16 & 1));
  const bool even = a.page.d % ROWS == 0;                   // whether those always share a page
  PageWindow pages(a, rt.req);
  const char* const kbase = (const char*)a.kc + (int64_t)kvh * a.page.d * (DIM * sizeof(E));
  const char* const vbase = (const char*)a.vc + (int64_t)kvh * a.page.d * (DIM * sizeof(E));

  // One tile of rows; by request, the further ones of a request that has more
  // than its hint said.
  for (int first = rt.first; first < rt.rows; first += BY_REQUEST ? 16 * RB : rt.rows) {
    const int rows = min(16 * RB, rt.rows - first);
    const int pa = pos0 + (int)fdiv(first, a.gdiv);
    const int pb = pos0 + (int)fdiv(first + rows - 1, a.gdiv);
    const KeyRange<KT> range(a, pa, pb, seq);
    int per;
    const int splits = split_of(range.tiles, a.splits, a.min_keys / KT, per);
    if (split >= splits) continue;
    const int t0 = split * per, nt = max(0, min(per, range.tiles - t0));

    // this lane's rows (the MFMA columns l16 of each block): their queries, zero
    // past the last row, and their positions
    u32x4v_t q[RB][QS];
    int qpos[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int r = 16 * b + l16;
      const int tok = (int)fdiv(first + r, a.gdiv);
      const int head = kvh * a.group + first + r - tok * a.group;
      qpos[b] = pos0 + tok;
      const bool in = r < rows;
      const u32x4v_t* src = reinterpret_cast<const u32x4v_t*>(
          (const E*)a.q + (in ? (int64_t)(rt.start + tok) * a.q_stride + head * DIM : 0));
#pragma unroll
      for (int s = 0; s < QS; ++s) q[b][s] = in ? src[4 * s + gq] : u32x4v_t{0, 0, 0, 0};
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
        const int key = t.base + l16;
        const int page = pages.at((int)fdiv(key, a.page));  // of every lane's key
        t.valid = (uint32_t)__ballot(range.has(key) && page >= 0) & ALL;
      }
      return t;
    };
    // Issues the DMA of its K rows or its V rows, or of both.
    auto issue = [&](const Tile& t, int stage, bool k, bool v) __attribute__((always_inline)) {
      uint4* const kt = my + stage * R::STAGE;
      uint4* const vt = kt + KT * P;
      if (even && t.valid == ALL) {
        // one page per instruction: the addresses are scalar work
        uint32_t ko = koff, vo = voff;
        asm volatile("" : "+v"(ko), "+v"(vo));  // or every x would keep its registers
#pragma unroll
        for (int x = 0; x < NI; ++x) {
          const int key = t.base + x * ROWS, pg = (int)fdiv(key, a.page);
          const int64_t off = key - pg * (int)a.page.d, page = pages.uniform_at(pg);
          // (the swizzles are linear: that of row r0 + x ROWS is r0's xor that of x ROWS)
          if (k)
            dma16(kbase + page * a.k_page + off * ROW, ko ^ 16 * kswz<P>(x * ROWS),
                  lds_addr(kt + 64 * x));
          if (v)
            dma16(vbase + page * a.v_page + off * ROW, vo ^ 16 * vswz<E, P>(x * ROWS),
                  lds_addr(vt + 64 * x));
        }
        return;
      }
#pragma unroll 1
      for (int x = 0; x < NI; ++x) {
        const int r = (64 * x + lane) / P, ps = lane % P, key = t.base + r;
        const int pg = (int)fdiv(key, a.page);
        const int64_t off = key - pg * (int)a.page.d, page = pages.at(pg);
        const char* kp = kbase + page * a.k_page + off * ROW + 16 * (ps ^ kswz<P>(r));
        const char* vp = vbase + page * a.v_page + off * ROW + 16 * (ps ^ vswz<E, P>(r));
        if (!((t.valid >> r) & 1)) kp = vp = (const char*)&attn_zero;
        if (k) dma16(kp, lds_addr(kt + 64 * x));
        if (v) dma16(vp, lds_addr(vt + 64 * x));
      }
    };

    // O += P V key by key on the vector unit, added where the key is visible: V may
    // hold infinities or NaN that some rows must not see (0 times them is NaN).
    auto by_key = [&](const Tile& t, const uint4* vt, const f32x4_t (&s)[RB]) {
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
          __builtin_amdgcn_sched_barrier(0);  // few registers at a time
          u32x4v_t v;
          if constexpr (R::F32) {
            v = __builtin_bit_cast(u32x4v_t, vt[j * P + ((4 * d + gq) ^ vswz<E, P>(j))]);
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(
                reinterpret_cast<const char*>(vt + j * P + ((2 * d + (gq >> 1)) ^ vswz<E, P>(j))) +
                8 * (gq & 1));
            v = u32x4v_t{__float_as_uint(Half<E>::widen(u.x & 0xffffu)),
                         __float_as_uint(Half<E>::widen(u.x >> 16)),
                         __float_as_uint(Half<E>::widen(u.y & 0xffffu)),
                         __float_as_uint(Half<E>::widen(u.y >> 16))};
          }
#pragma unroll
          for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[d][b][i] = fmaf(p[b], __uint_as_float(v[i] & see[b]), o[d][b][i]);
        }
      }
    };

    f32x4_t s[RB];
    auto scores = [&](int stage) __attribute__((always_inline)) {  // S^T = K Q^T
      uint32_t at = ka + stage * (R::STAGE * 16);
      asm volatile("" : "+v"(at));  // or every step would keep its address
#pragma unroll
      for (int b = 0; b < RB; ++b) s[b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < QS; ++i) {
        const u32x4v_t kf = lds_read16(at ^ 64 * i);
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          if constexpr (R::F32) {
            const f32x4_t x = __builtin_bit_cast(f32x4_t, kf);
            const f32x4_t y = __builtin_bit_cast(f32x4_t, q[b][i]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], y[e], s[b], 0, 0, 0);
          } else {
            typedef typename Half<E>::frag frag;
            s[b] = Half<E>::mma16(__builtin_bit_cast(frag, kf), __builtin_bit_cast(frag, q[b][i]), s[b]);
          }
        }
      }
    };
    // The softmax of the tile's scores, and `values` before V is read.
    // CAREFUL keeps the values of hidden keys out of the sums.
    auto weigh = [&](auto careful, const Tile& t, int stage, auto values) __attribute__((always_inline)) {
      constexpr bool CAREFUL = decltype(careful)::value;
      const uint4* const vt = my + stage * R::STAGE + KT * P;
      // keys hidden from some rows, or absent
      const bool mixed = pa != pb && (t.base + KT - 1 > pa ||
                                      (a.window > 0 && t.base <= pb - a.window && t.base + KT > a.sinks));
      if (mixed || t.valid != ALL) {
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          const uint32_t see = seen(a, t.base, qpos[b], t.valid) >> (4 * gq);
#pragma unroll
          for (int r = 0; r < 4; ++r) s[b][r] = see & (1u << r) ? s[b][r] : NEG_INF;
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
        const float mb = (m[b] == NEG_INF ? 0.0f : m[b]) - BIAS;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float p = exp2_fast(fmaf(s[b][r], c, -mb));
          s[b][r] = p;
          l[b] += p;
        }
      }
      values();
      if constexpr (CAREFUL) {
        if (mixed) {
          by_key(t, vt, s);
          return;
        }
      }
      if constexpr (R::F32) {
        uint32_t at = va + stage * (R::STAGE * 16);
        asm volatile("" : "+v"(at));
#pragma unroll
        for (int d = 0; d < DIM / 16; ++d) {
          if (d % 2 == 0) __builtin_amdgcn_sched_barrier(0);  // few registers at a time
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = lds_read4((at ^ 64 * d) + e * ROW);
#pragma unroll
            for (int b = 0; b < RB; ++b)
              o[d][b] = __builtin_amdgcn_mfma_f32_16x16x4f32(x, s[b][e], o[d][b], 0, 0, 0);
          }
        }
      } else {
        // P^T as it lies: lane group gq holds keys 4 gq + r
        typename Half<E>::quad p[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int r = 0; r < 4; ++r) Half<E>::set(p[b], r, s[b][r]);
        const uint32_t at = va + stage * (R::STAGE * 16);
#pragma unroll
        for (int d = 0; d < DIM / 16; ++d) {
          const s16x4_t v = lds_read_tr(at ^ 32 * d);
#pragma unroll
          for (int b = 0; b < RB; ++b) o[d][b] = Half<E>::mma16k16(v, p[b], o[d][b]);
        }
      }
    };

    // contiguous tiles per wave
    const int share = (nt + WAVES - 1) / WAVES;
    const int w0 = t0 + min(nt, wave * share), w1 = t0 + min(nt, (wave + 1) * share);
    auto walk = [&](auto careful) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        m[b] = NEG_INF;
        l[b] = 0.0f;
#pragma unroll
        for (int d = 0; d < DIM / 16; ++d) o[d][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
      if (w0 >= w1) return;
      Tile cur = locate(w0);
      if constexpr (R::STAGES == 2) {
        issue(cur, 0, true, true);
      } else {
        issue(cur, 0, true, false);
        issue(cur, 0, false, true);
      }
      // the queries arrive here: a wait for them in the loop would wait for the DMA too
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int x = 0; x < QS; ++x) asm volatile("" : "+v"(q[b][x]));
#pragma unroll 1
      for (int i = w0; i < w1; ++i) {
        const bool more = i + 1 < w1;
        Tile next = cur;
        if constexpr (R::STAGES == 2) {
          const int stage = (i - w0) & 1;
          if (more) {
            lds_wait();  // the reads of the tile that this one replaces
            next = locate(i + 1);
            issue(next, stage ^ 1, true, true);
            dma_wait<2 * NI>();
          } else {
            dma_wait<0>();
          }
          scores(stage);
          weigh(careful, cur, stage, [] {});
        } else {
          dma_wait<NI>();  // K of this tile; V may still be on its way
          scores(0);
          lds_wait();
          if (more) {
            next = locate(i + 1);
            issue(next, 0, true, false);
          }
          weigh(careful, cur, 0, [&] {
            if (more) dma_wait<NI>();
            else dma_wait<0>();
          });
          lds_wait();
          if (more) issue(next, 0, false, true);
        }
        cur = next;
      }
    };
    walk(std::false_type{});
    if (pa != pb) {  // else every key of a tile is visible to all rows
      // a hidden infinity or NaN of V has spoilt the sums of its tile: once more, carefully
      float z = 0.0f;  // becomes NaN if any sum is not finite
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int d = 0; d < DIM / 16; ++d)
#pragma unroll
          for (int r = 0; r < 4; ++r) z = fmaf(o[d][b][r], 0.0f, z);
      if (__any(z != 0.0f)) {
        lds_wait();
        walk(std::true_type{});
      }
    }

    // join of the four waves
#pragma unroll
    for (int b = 0; b < RB; ++b) l[b] = sum_quarter(l[b]);
    __syncthreads();
    float* const so = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int r = 16 * b + l16;
      if (gq == 0) {
        sm_m[wave][r] = m[b];
        sm_l[wave][r] = l[b];
      }
#pragma unroll
      for (int d = 0; d < DIM / 16; ++d)
        *reinterpret_cast<f32x4_t*>(so + (wave * 16 * RB + r) * R::OS + 16 * d + 4 * gq) = o[d][b];
    }
    __syncthreads();
    constexpr int PER = DIM / 4;  // threads per row
    for (int x = threadIdx.x; x < rows * PER; x += 64 * WAVES) {
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
        const f32x4_t y = *reinterpret_cast<const f32x4_t*>(so + (w * 16 * RB + r) * R::OS + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(f, y[i], acc[i]);
      }
      // a row that sees no key has sum 0: zeros, and a log-sum-exp of -inf
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = sum == 0.0f ? 0.0f : acc[i] * inv;
      const float lse2 = sum == 0.0f ? NEG_INF : base - BIAS + __log2f(sum);
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
    if (BY_REQUEST) __syncthreads();  // before the next tile's DMA
  }
}

// The join of a row's splits, in their order:
// out = sum_s 2^(lse_s - top) O_s / sum_s 2^(lse_s - top).
// Lane s weighs split s (there are at most 64): the weight, and what the weights sum to.
__device__ __forceinline__ float split_weight(float e, float& base, float& sum) {
  float top = e;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  base = top == NEG_INF ? 0.0f : top;
  const float f = exp2_fast(e - base);
  sum = f;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  return f;
}
__device__ __forceinline__ float lane_value(float x, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), lane));
}

template <typename E, int DIM>
__device__ __forceinline__ void join_store(const AttnLaunch& a, int64_t row, const float* acc, float base,
                                           float sum, int lane) {
  constexpr int V = DIM / 64;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  E* dst = (E*)a.out + row * DIM + V * lane;
#pragma unroll
  for (int i = 0; i < V; ++i) dst[i] = from_f32<E>(acc[i] * inv);
  if (a.lse != nullptr && lane == 0)
    a.lse[row] = sum == 0.0f ? NEG_INF : (base + __log2f(sum)) * LN2;
}

// Few rows: four waves share one, a quarter of the splits each.  Bound by latency, so
// nothing waits for the number of splits but the sums: all loads go out at once.
template <typename E, int DIM> __global__ __launch_bounds__(256) void join_few_kernel(const AttnLaunch a) {
  constexpr int V = DIM / 64, AT_ONCE = 16;
  __shared__ float sm[4][DIM];
  const int lane = threadIdx.x & 63, wave = wave_of();
  const int64_t rows = (int64_t)a.total * a.hq, row = blockIdx.x;
  const int cut = a.part_n[row], c0 = a.cu[0], c1 = a.cu[a.n];
  float e = lane < a.splits ? a.part_lse[lane * rows + row] : NEG_INF;
  const float* src = a.part_o + row * DIM + V * lane;
  float x[AT_ONCE][V];
#pragma unroll
  for (int j = 0; j < AT_ONCE; ++j) {
    const int s = min(16 * wave + j, a.splits - 1);
#pragma unroll
    for (int i = 0; i < V; ++i) x[j][i] = src[s * rows * DIM + i];
  }
  // only rows of the batch that were split
  const int64_t first = (int64_t)min(max(c0, 0), a.total) * a.hq;
  const int64_t last = (int64_t)min(max(c1, 0), a.total) * a.hq;
  if (row < first || row >= last || cut <= 1) return;
  const int n = min(cut, a.splits);
  if (lane >= n) e = NEG_INF;
  float base, sum, acc[V] = {};
  const float f = split_weight(e, base, sum);
#pragma unroll
  for (int j = 0; j < AT_ONCE; ++j) {
    const int s = 16 * wave + j;
    const float g = lane_value(f, s);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = s < n ? fmaf(g, x[j][i], acc[i]) : acc[i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) sm[wave][V * lane + i] = acc[i];
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < 4; ++w)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += sm[w][V * lane + i];
  join_store<E, DIM>(a, row, acc, base, sum, lane);
}

// Many rows, some of which were not split: 16 lanes share one.  The partials are asked
// for with their lse, eight splits at a time.
template <typename E, int DIM> __global__ __launch_bounds__(256) void join_kernel(const AttnLaunch a) {
  constexpr int V = DIM / 16, AT_ONCE = 8;
  const int lane = threadIdx.x & 63, at = lane & 15;
  const int64_t rows = (int64_t)a.total * a.hq;
  const int64_t row = ((int64_t)blockIdx.x * 4 + wave_of()) * 4 + (lane >> 4);
  const int64_t first = (int64_t)min(max(a.cu[0], 0), a.total) * a.hq;
  const int64_t last = (int64_t)min(max(a.cu[a.n], 0), a.total) * a.hq;
  const int cut = row >= first && row < last ? a.part_n[row] : 1;
  const int n = cut > 1 ? min(cut, a.splits) : 0;
  if (n == 0) return;  // a row's 16 lanes leave together
  const float* src = a.part_o + row * DIM + V * at;
  float x[AT_ONCE][V];
  auto load = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j)
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 f = *(const float4*)(src + min(s + j, n - 1) * rows * DIM + i);
        x[j][i] = f.x, x[j][i + 1] = f.y, x[j][i + 2] = f.z, x[j][i + 3] = f.w;
      }
  };
  // lane i weighs the splits i, i + 16, i + 32 and i + 48
  float f[4], top = NEG_INF, sum = 0.0f, acc[V] = {};
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = at + 16 * k < n ? a.part_lse[(at + 16 * k) * rows + row] : NEG_INF;
  load(0);
#pragma unroll
  for (int k = 0; k < 4; ++k) top = fmaxf(top, f[k]);
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  const float base = top == NEG_INF ? 0.0f : top;
#pragma unroll
  for (int k = 0; k < 4; ++k) sum += f[k] = exp2_fast(f[k] - base);
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  for (int s = 0;;) {
    const float w = s < 16 ? f[0] : s < 32 ? f[1] : s < 48 ? f[2] : f[3];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      const float g = __shfl(w, (s & 15) + j, 16);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = s + j < n ? fmaf(g, x[j][i], acc[i]) : acc[i];
    }
    s += AT_ONCE;
    if (s >= n) break;
    load(s);
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < V; i += 4)
    store4((E*)a.out + row * DIM + V * at + i, acc[i] * inv, acc[i + 1] * inv, acc[i + 2] * inv,
           acc[i + 3] * inv);
  if (a.lse != nullptr && at == 0)
    a.lse[row] = sum == 0.0f ? NEG_INF : (base + __log2f(sum)) * LN2;
}

template <typename E, int DIM, int RB> hipError_t rows_go(const AttnLaunch& L) {
  if (L.by_request) {
    hipLaunchKernelGGL((rows_kernel<E, DIM, RB, true>),
                       dim3((unsigned)(L.n * L.hkv), (unsigned)L.splits), dim3(64 * WAVES), 0,
                       (hipStream_t)L.stream, L);
  } else if constexpr (sizeof(E) == 4 && RB == 2) {  // the only one that is asked for
    const int64_t tiles = (int64_t)L.total * L.group / (16 * RB) + L.n;
    hipLaunchKernelGGL((rows_kernel<E, DIM, RB, false>),
                       dim3((unsigned)(tiles * L.hkv), (unsigned)L.splits), dim3(64 * WAVES), 0,
                       (hipStream_t)L.stream, L);
  }
  return hipGetLastError();
}
template <typename E, int DIM> hipError_t rows_rb(const AttnLaunch& L) {
  return L.row_blocks == 1 ? rows_go<E, DIM, 1>(L) : rows_go<E, DIM, 2>(L);
}
template <typename E> hipError_t rows_dim(const AttnLaunch& L) {
  return L.dim == 64 ? rows_rb<E, 64>(L) : rows_rb<E, 128>(L);
}

template <typename E, int DIM> hipError_t join_go(const AttnLaunch& L) {
  const int64_t rows = (int64_t)L.total * L.hq;
  if (rows * L.splits <= 16384) {  // reads every split's place, used or not: 8 MB at most
    hipLaunchKernelGGL((join_few_kernel<E, DIM>), dim3((unsigned)rows), dim3(256), 0,
                       (hipStream_t)L.stream, L);
  } else {
    hipLaunchKernelGGL((join_kernel<E, DIM>), dim3((unsigned)((rows + 15) / 16)), dim3(256), 0,
                       (hipStream_t)L.stream, L);
  }
  return hipGetLastError();
}
template <typename E> hipError_t join_dim(const AttnLaunch& L) {
  return L.dim == 64 ? join_go<E, 64>(L) : join_go<E, 128>(L);
}

}  // namespace

hipError_t launch_attn_rows(const AttnLaunch& L) {
  switch (L.dtype) {
    case 0: return rows_dim<float>(L);
    case 1: return rows_dim<bf16>(L);
    default: return rows_dim<_Float16>(L);
  }
}

hipError_t launch_attn_join(const AttnLaunch& L) {
  switch (L.dtype) {
    case 0: return join_dim<float>(L);
    case 1: return join_dim<bf16>(L);
    default: return join_dim<_Float16>(L);
  }
}

}  // namespace kda
