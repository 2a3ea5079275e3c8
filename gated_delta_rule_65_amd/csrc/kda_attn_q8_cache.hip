// Rows into and out of the paged cache in 8 bits (kda_paged_q8.h).
//
// Append.  A block's scale follows the largest magnitude among its new rows, and its
// earlier rows where it already has some, so the unit of work is (block, head): a wave, or
// two or four of them where blocks are long, hold the block's new rows in registers, take their
// largest magnitude, settle the scale and write the codes.  No block belongs to two units, so
// there are no atomics, and the rows are read once.  Request i's units start at
// floor(cu[i] / block) + 2 i, which leaves it as many as its rows can touch.  Bound by HBM
// where rows are many: 30669 tokens of 8 heads of 128 bf16 channels (126 MB in, 63 MB out) 46 us,
// 4.1 TB/s, in blocks of 8 (44 us), 16, 32 (one wave a block: 51 us, four: 59) or 64.  Smaller blocks
// leave lanes idle and pay each unit's search and trips for fewer rows (blocks of 4: 56 us, a scale per token:
// 190); in longer ones the rows past the registers are loaded twice by few units (128: 63 us, 256: 69,
// 512: 78).  By latency where rows are few: 256 requests of one token 6 us, three round trips to memory
// (offsets and lengths; the rows and the table's entry; the old scale) and the writes; in blocks of
// 512 whose earlier rows are rounded anew 6 us more.
//
// Read.  Units of four consecutive rows of one request; each thread widens the codes of 16
// bytes of output, which a wave's stores join to whole lines.  30935 rows as fp32 (63 MB in, 253
// out) 55 us, 5.8 TB/s; as bf16 51 us for 49385 rows, 5.9 TB/s; with 8 codes to a thread also in
// fp32 66 us, with units of 16 rows 76, with stores past the caches 132.
#include "kda_attn_q8.hpp"

namespace kda {
namespace {

// 8 values of a row.
template <typename E> struct Eight;
template <> struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p) {
    a = ((const float4*)p)[0];
    b = ((const float4*)p)[1];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
template <typename E> struct Eight {
  uint4 u;
  __device__ __forceinline__ void load(const void* p) { u = *(const uint4*)p; }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = Half<E>::widen(w[i] & 0xffffu);
      x[2 * i + 1] = Half<E>::widen(w[i] >> 16);
    }
  }
};

// The largest finite magnitude.
__device__ __forceinline__ float top_of(const float (&x)[8], float top) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = fabsf(x[i]);
    top = fmaxf(top, y < __builtin_inff() ? y : 0.0f);
  }
  return top;
}
template <int CODE> __device__ __forceinline__ uint2 encode8(const float (&x)[8], float f) {
  const float a[4] = {x[0] * f, x[1] * f, x[2] * f, x[3] * f};
  const float b[4] = {x[4] * f, x[5] * f, x[6] * f, x[7] * f};
  return make_uint2(Code<CODE>::encode(a), Code<CODE>::encode(b));
}
__device__ __forceinline__ float max_wave(float x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x = fmaxf(x, __shfl_xor(x, d));
  return x;
}

// The scale of a block that has rows; one that is no finite number becomes NaN, which is neither the larger
// of two nor less than another.
__device__ __forceinline__ float begun_scale(float s) {
  return fabsf(s) < __builtin_inff() ? pow2_scale(s) : __builtin_nanf("");
}

// WAVES: waves that share a block.
template <typename E, int DIM, int CODE, int WAVES>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void append_q8_kernel(const CacheQ8Launch a, uint32_t units) {
  constexpr int LPR = DIM / 8, RPL = 64 / LPR * WAVES;  // lanes per row, rows per step
  constexpr int HOLD = 4;                               // steps held in registers
  __shared__ float s_top[2][WAVES];
  const int lane = threadIdx.x & 63, wave = wave_of();
  const uint32_t w = WAVES == 1 ? blockIdx.x * 4 + wave : blockIdx.x;
  if (w >= units) return;
  const uint32_t item = fdiv(w, a.hdiv);
  const int head = (int)(w - item * a.hkv);
  auto first_item = [&](int i, int start) { return (int)fdiv(start, a.block) + 2 * i; };
  const Rows own = find_rows(a.cu, a.seq, a.n, a.total, (int)item, lane, first_item);
  const int req = own.req, start = own.start, len = own.len;
  const int64_t seq = own.seq, pos0 = seq - len;
  const int local = (int)item - first_item(req, start);
  if (local < 0) return;  // offsets that decrease
  // the block, among those of the request, and its new rows
  const int B = (int)a.block.d;
  const int64_t bi = (int64_t)fdiv((uint32_t)max(pos0, (int64_t)0), a.block) + local, at = bi * B;
  const int64_t lo = max(pos0, at), hi = min(min(seq, a.capacity), at + B);
  if (lo >= hi) return;
  const int page_at = (int)fdiv((uint32_t)at, a.page);  // at < capacity
  const int id = a.table[(int64_t)req * a.table_stride + page_at];
  const int rows = (int)(hi - lo), held = (int)(lo - at);

  const int first = (WAVES == 1 ? 0 : wave * (64 / LPR)) + lane / LPR, col = 8 * (lane % LPR);
  const int64_t x0 = start + (lo - pos0);
  const char* const kin = (const char*)a.k + x0 * a.k_stride + ((int64_t)head * DIM + col) * sizeof(E);
  const char* const vin = (const char*)a.v + x0 * a.v_stride + ((int64_t)head * DIM + col) * sizeof(E);
  Eight<E> k[HOLD], v[HOLD];
  auto load = [&](int r0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < HOLD; ++i) {
      const int r = r0 + i * RPL + first;
      if (r < rows) {
        k[i].load(kin + r * a.k_stride);
        v[i].load(vin + r * a.v_stride);
      }
    }
  };
  load(0);  // beside the table's entry, which only the codes' place needs
  if ((uint32_t)id >= (uint32_t)a.num_pages) return;
  const int off = (int)at - page_at * (int)a.page.d;  // of the block in its page
  const int64_t row_at = ((int64_t)head * a.page.d + off) * DIM;
  uint8_t* const kc = (uint8_t*)a.kc + id * a.k_page + row_at;
  uint8_t* const vc = (uint8_t*)a.vc + id * a.v_page + row_at;
  const int64_t sc = ((int64_t)id * a.hkv + head) * a.per_page + fdiv(off, a.block);
  const float ks0 = held > 0 ? begun_scale(a.ks[sc]) : 0.0f, vs0 = held > 0 ? begun_scale(a.vs[sc]) : 0.0f;
  float ktop = 0.0f, vtop = 0.0f;
  for (int r0 = 0; r0 < rows; r0 += HOLD * RPL) {
    if (r0 > 0) load(r0);
#pragma unroll
    for (int i = 0; i < HOLD; ++i)
      if (r0 + i * RPL + first < rows) {
        float x[8];
        k[i].get(x);
        ktop = top_of(x, ktop);
        v[i].get(x);
        vtop = top_of(x, vtop);
      }
  }
  ktop = max_wave(ktop);
  vtop = max_wave(vtop);
  if constexpr (WAVES > 1) {
    if (lane == 0) {
      s_top[0][wave] = ktop;
      s_top[1][wave] = vtop;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      ktop = fmaxf(ktop, s_top[0][i]);
      vtop = fmaxf(vtop, s_top[1][i]);
    }
  }
  const float ks = fmaxf(Code<CODE>::least_scale(ktop), ks0);
  const float vs = fmaxf(Code<CODE>::least_scale(vtop), vs0);
  const float kf = inverse_scale(ks), vf = inverse_scale(vs);
  for (int r0 = 0; r0 < rows; r0 += HOLD * RPL) {
    if (rows > HOLD * RPL) load(r0);
#pragma unroll
    for (int i = 0; i < HOLD; ++i) {
      const int r = r0 + i * RPL + first;
      if (r < rows) {
        float x[8];
        k[i].get(x);
        *(uint2*)(kc + (int64_t)(held + r) * DIM + col) = encode8<CODE>(x, kf);
        v[i].get(x);
        *(uint2*)(vc + (int64_t)(held + r) * DIM + col) = encode8<CODE>(x, vf);
      }
    }
  }
  // earlier rows of a block whose scale grew
  auto shrink = [&](uint8_t* c, float f) __attribute__((always_inline)) {
    for (int r = first; r < held; r += RPL) {
      uint2* const p = (uint2*)(c + (int64_t)r * DIM + col);
      const uint2 u = *p;
      float x[4], y[4];
      Code<CODE>::widen(u.x, x);
      Code<CODE>::widen(u.y, y);
      const float z[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
      *p = encode8<CODE>(z, f);
    }
  };
  if (held > 0 && ks > ks0) shrink(kc, ks0 * kf);
  if (held > 0 && vs > vs0) shrink(vc, vs0 * vf);
  if (lane == 0 && (WAVES == 1 || wave == 0)) {
    a.ks[sc] = ks;
    a.vs[sc] = vs;
  }
}

// A thread's 16 bytes of a row: the values of 4 or 8 codes.
template <typename E, int CODE> struct Out {
  static constexpr int N = 16 / (int)sizeof(E);
  uint32_t u[N / 4];
  float s;
  __device__ __forceinline__ void load(const uint8_t* p, const float* scale) {
    if constexpr (N == 4) {
      u[0] = *(const uint32_t*)p;
    } else {
      const uint2 w = *(const uint2*)p;
      u[0] = w.x, u[1] = w.y;
    }
    s = *scale;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) u[i] = 0;
    s = 0.0f;
  }
  __device__ __forceinline__ void store(E* p) const {
    float z = s;
    asm volatile("" : "+v"(z));  // or the mask moves to the load and waits for it there: 53 us for 50
    z = pow2_scale(z);
    float x[N];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      float y[4];
      Code<CODE>::widen(u[i], y);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[4 * i + j] = y[j] * z;
    }
    if constexpr (N == 4) {
      store4(p, x[0], x[1], x[2], x[3]);
    } else {
      typename Half<E>::frag f;
#pragma unroll
      for (int i = 0; i < 8; ++i) Half<E>::set(f, i, x[i]);
      *reinterpret_cast<typename Half<E>::frag*>(p) = f;
    }
  }
};

// Rows of a unit: few, so that a small call has many units and few loads per thread.
constexpr int READ_ROWS = 4;

template <typename E, int DIM, int CODE>
__global__ __launch_bounds__(256) void read_q8_kernel(const CacheQ8Launch a, FastDiv per_token) {
  typedef Out<E, CODE> Piece;
  constexpr int LPR = DIM / Piece::N;
  __shared__ int64_t s_k[READ_ROWS], s_v[READ_ROWS], s_s[READ_ROWS];  // bytes, bytes, scales; -1: no page
  const int tid = threadIdx.x, lane = tid & 63;
  const int item = (int)blockIdx.x;
  const Rows own = find_rows(a.cu, a.seq, a.n, a.total, item, lane,
                             [&](int i, int start) { return start / READ_ROWS + i; });
  const int req = own.req, start = own.start, len = own.len;
  const int first = (item - (start / READ_ROWS + req)) * READ_ROWS;
  if (first < 0 || first >= len) return;
  const int rows = min(READ_ROWS, len - first);
  if (tid < rows) {
    const int64_t pos = (int64_t)own.seq - len + first + tid;
    int64_t kb = -1, vb = -1, sb = 0;
    if (pos >= 0 && pos < a.capacity) {
      const int pg = (int)fdiv((uint32_t)pos, a.page), off = (int)pos - pg * (int)a.page.d;
      const int id = a.table[(int64_t)req * a.table_stride + pg];
      if ((uint32_t)id < (uint32_t)a.num_pages) {
        kb = id * a.k_page + (int64_t)off * DIM;
        vb = id * a.v_page + (int64_t)off * DIM;
        sb = (int64_t)id * a.hkv * a.per_page + fdiv(off, a.block);
      }
    }
    s_k[tid] = kb, s_v[tid] = vb, s_s[tid] = sb;
  }
  __syncthreads();
  const int64_t head = (int64_t)a.page.d * DIM;  // bytes between heads
  const uint32_t total = rows * per_token.d;
  // AT_ONCE steps' loads go out together: a few rows are bound by latency
  constexpr int AT_ONCE = 4;
  for (uint32_t x0 = tid; x0 < total; x0 += 256 * AT_ONCE) {
    Piece k[AT_ONCE], v[AT_ONCE];
    int64_t to[AT_ONCE];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      const uint32_t x = x0 + 256 * j;
      k[j].zero();
      v[j].zero();
      if (x < total) {
        const uint32_t t = fdiv(x, per_token), p = x - t * per_token.d;
        const int h = (int)(p / LPR), col = Piece::N * (int)(p % LPR);
        to[j] = (int64_t)(start + first + (int)t) * a.hkv * DIM + Piece::N * (int64_t)p;
        const int64_t kb = s_k[t], at = s_s[t] + (int64_t)h * a.per_page;
        if (kb >= 0) {
          k[j].load((const uint8_t*)a.kc + kb + h * head + col, a.ks + at);
          v[j].load((const uint8_t*)a.vc + s_v[t] + h * head + col, a.vs + at);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      if (x0 + 256 * j >= total) break;
      k[j].store((E*)a.ko + to[j]);
      v[j].store((E*)a.vo + to[j]);
    }
  }
}

template <typename E, int DIM, int CODE> hipError_t append_go(const CacheQ8Launch& L) {
  const uint32_t items = (uint32_t)L.total / L.block.d + 2u * (uint32_t)L.n;
  const uint32_t units = items * (uint32_t)L.hkv;
  const hipStream_t stream = (hipStream_t)L.stream;
  // as many waves as hold a block's rows (128 channels) in their registers, four at most (times of blocks of 1
  // to 512 above)
  if (L.block.d <= 16)
    hipLaunchKernelGGL((append_q8_kernel<E, DIM, CODE, 1>), dim3((units + 3) / 4), dim3(256), 0, stream, L, units);
  else if (L.block.d <= 32)
    hipLaunchKernelGGL((append_q8_kernel<E, DIM, CODE, 2>), dim3(units), dim3(128), 0, stream, L, units);
  else
    hipLaunchKernelGGL((append_q8_kernel<E, DIM, CODE, 4>), dim3(units), dim3(256), 0, stream, L, units);
  return hipGetLastError();
}
template <typename E, int DIM, int CODE> hipError_t read_go(const CacheQ8Launch& L) {
  const uint32_t items = (uint32_t)(L.total / READ_ROWS) + (uint32_t)L.n;
  hipLaunchKernelGGL((read_q8_kernel<E, DIM, CODE>), dim3(items), dim3(256), 0, (hipStream_t)L.stream, L,
                     fast_div((uint32_t)(L.hkv * DIM / Out<E, CODE>::N)));
  return hipGetLastError();
}

template <typename E, int DIM> hipError_t append_code(const CacheQ8Launch& L) {
  return L.code == E4M3 ? append_go<E, DIM, E4M3>(L) : append_go<E, DIM, INT8>(L);
}
template <typename E> hipError_t append_dim(const CacheQ8Launch& L) {
  return L.dim == 64 ? append_code<E, 64>(L) : append_code<E, 128>(L);
}
template <typename E, int DIM> hipError_t read_code(const CacheQ8Launch& L) {
  return L.code == E4M3 ? read_go<E, DIM, E4M3>(L) : read_go<E, DIM, INT8>(L);
}
template <typename E> hipError_t read_dim(const CacheQ8Launch& L) {
  return L.dim == 64 ? read_code<E, 64>(L) : read_code<E, 128>(L);
}

}  // namespace

hipError_t launch_append_q8(const CacheQ8Launch& L) {
  switch (L.dtype) {
    case 0: return append_dim<float>(L);
    case 1: return append_dim<bf16>(L);
    default: return append_dim<_Float16>(L);
  }
}

hipError_t launch_read_q8(const CacheQ8Launch& L) {
  switch (L.dtype) {
    case 0: return read_dim<float>(L);
    case 1: return read_dim<bf16>(L);
    default: return read_dim<_Float16>(L);
  }
}

}  // namespace kda
