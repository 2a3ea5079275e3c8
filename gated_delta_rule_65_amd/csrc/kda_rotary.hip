// Rotary positions of query and key rows (kda_rotary.h): the kernel and its C-ABI entry.
//
// A pair of channels turns by position times frequency.  The angle is formed in fp64 in
// turns and brought to half a turn either way, so that far positions lose nothing; its
// sine and cosine are fp32.  A workgroup computes the sines and cosines of a few tokens
// once, in LDS, and then streams the tokens' heads past them.
//
// Bound by HBM where tokens are many: 32768 of 40 heads of 128 fp16 channels (336 MB in and
// out) 127 us, 5.3 TB/s, where a large copy reaches 5.2; by latency where they are few (256
// tokens 3.6 us), so few tokens have a workgroup each, many share one by four.
//
// Channels go in pieces of 16 bytes where the pairs fill them, else one by one, which is bound by the
// vector unit (77 % busy): 32768 of 40 heads of 128 in fp16 with 64, 32 or 20 interleaved
// pairs 125, 130 and 137 us; with 20, 27 or 63 pairs as halves 378, 374 and 285 us, with 27
// interleaved 368 us.
#include <math.h>

#include <cmath>

#include "../../include/kda_rotary.h"
#include "kda_common.hpp"
#include "kda_paged.hpp"

#define KDA_API extern "C" __attribute__((visibility("default")))
#define FAIL(status, ...) return (kda_status)kda::set_error(status, __VA_ARGS__)

namespace kda {
namespace {

constexpr int MAX_DIM = 512, MAX_TB = 4;
constexpr int64_t MAX_GROUPS = ((int64_t)1 << 24) - 1;  // of 256: a launch holds fewer than 2^32 threads

struct RotaryLaunch {
  const void *q, *k;
  void *qo, *ko;
  const int32_t* pos;
  const double* freq;
  int64_t tokens;
  int64_t qs, ks, qos, kos;  // elements between tokens
  int hq, heads, dim, n;     // heads of q and k; n pairs
  int turns, units;          // pieces of a head that turn, and all of them
  int tb;                    // tokens per workgroup
  FastDiv by_units, by_heads, by_n;
  float scale, sign;
};

__device__ __forceinline__ uint32_t rdiv(uint32_t t, const FastDiv& f) {
  return __umulhi(2u * t, f.mul) >> f.shift;
}

// 16 bytes of a row as floats.
template <typename E> struct Piece {
  static constexpr int V = 16 / (int)sizeof(E);
  E x[V];
};
template <typename E> __device__ __forceinline__ Piece<E> load_piece(const E* p) {
  return __builtin_bit_cast(Piece<E>, *reinterpret_cast<const uint4*>(p));
}
template <typename E> __device__ __forceinline__ void store_piece(E* p, const Piece<E>& v) {
  *reinterpret_cast<uint4*>(p) = __builtin_bit_cast(uint4, v);
}

template <typename E, bool INTER, bool WIDE>
__global__ __launch_bounds__(256) void rotary_kernel(const RotaryLaunch a) {
  constexpr int V = Piece<E>::V;
  __shared__ float2 cs[MAX_TB * MAX_DIM / 2];
  __shared__ int s_pos[MAX_TB];
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * a.tb;
  const int nt = (int)min((int64_t)a.tb, a.tokens - t0);
  for (int i = tid; i < nt * a.n; i += 256) {
    const int t = (int)rdiv(i, a.by_n), j = i - t * a.n;
    const int pos = a.pos[t0 + t];
    if (j == 0) s_pos[t] = pos;
    const double turns = (double)pos * (a.freq[j] * 0.15915494309189535);
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    cs[i] = make_float2(a.scale * c, a.sign * s);
  }
  __syncthreads();
  const uint32_t total = (uint32_t)nt * a.heads * a.units;
  for (uint32_t x = tid; x < total; x += 256) {
    const uint32_t row = rdiv(x, a.by_units), u = x - row * a.units;
    const uint32_t t = rdiv(row, a.by_heads);
    int h = (int)(row - t * a.heads);
    if (s_pos[t] < 0) continue;
    const bool is_q = h < a.hq;
    if (!is_q) h -= a.hq;
    const E* src = (const E*)(is_q ? a.q : a.k) + (t0 + t) * (is_q ? a.qs : a.ks) + (int64_t)h * a.dim;
    E* dst = (E*)(is_q ? a.qo : a.ko) + (t0 + t) * (is_q ? a.qos : a.kos) + (int64_t)h * a.dim;
    const float2* w = cs + t * a.n;
    if ((int)u >= a.turns) {  // channels that pass
      if (src == dst) continue;
      const int c = 2 * a.n + (int)(u - a.turns) * (WIDE ? V : 1);
      if constexpr (WIDE) store_piece(dst + c, load_piece(src + c));
      else dst[c] = src[c];
      continue;
    }
    if constexpr (!WIDE) {
      const int c0 = INTER ? 2 * u : u, c1 = INTER ? 2 * u + 1 : u + a.n;
      const float p = to_f32(src[c0]), r = to_f32(src[c1]);
      const float2 z = w[u];
      dst[c0] = from_f32<E>(p * z.x - r * z.y);
      dst[c1] = from_f32<E>(p * z.y + r * z.x);
    } else if constexpr (INTER) {
      const int c = V * u;
      Piece<E> v = load_piece(src + c);
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float p = to_f32(v.x[i]), r = to_f32(v.x[i + 1]);
        const float2 z = w[(c + i) / 2];
        v.x[i] = from_f32<E>(p * z.x - r * z.y);
        v.x[i + 1] = from_f32<E>(p * z.y + r * z.x);
      }
      store_piece(dst + c, v);
    } else {
      const int c = V * u;
      Piece<E> v0 = load_piece(src + c), v1 = load_piece(src + c + a.n);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float p = to_f32(v0.x[i]), r = to_f32(v1.x[i]);
        const float2 z = w[c + i];
        v0.x[i] = from_f32<E>(p * z.x - r * z.y);
        v1.x[i] = from_f32<E>(p * z.y + r * z.x);
      }
      store_piece(dst + c, v0);
      store_piece(dst + c + a.n, v1);
    }
  }
}

template <typename E> void rotary_go(const RotaryLaunch& L, bool inter, bool wide, hipStream_t stream) {
  const dim3 grid((unsigned)((L.tokens + L.tb - 1) / L.tb)), block(256);
  if (inter && wide) hipLaunchKernelGGL((rotary_kernel<E, true, true>), grid, block, 0, stream, L);
  else if (inter) hipLaunchKernelGGL((rotary_kernel<E, true, false>), grid, block, 0, stream, L);
  else if (wide) hipLaunchKernelGGL((rotary_kernel<E, false, true>), grid, block, 0, stream, L);
  else hipLaunchKernelGGL((rotary_kernel<E, false, false>), grid, block, 0, stream, L);
}

// A set of rows in memory.
struct RowSet {
  uintptr_t at;
  int64_t row, stride;  // bytes of a row, between rows
};
bool share(const RowSet& a, const RowSet& b, int64_t rows) {
  if (a.at >= b.at + (uintptr_t)((rows - 1) * b.stride + b.row) ||
      b.at >= a.at + (uintptr_t)((rows - 1) * a.stride + a.row))
    return false;
  if (a.stride != b.stride) return true;  // as far as anyone looks
  // columns of one wider array: apart if they are apart modulo its row
  const int64_t d = (int64_t)(b.at - a.at) % a.stride, gap = d < 0 ? d + a.stride : d;
  return gap < a.row || a.stride - gap < b.row;
}

}  // namespace
}  // namespace kda

KDA_API kda_status kda_rotary(const kda_rotary_args* a) {
  using namespace kda;
  if (!a) FAIL(KDA_ERR_ARG, "args is NULL");
  if (a->struct_size != sizeof(kda_rotary_args))
    FAIL(KDA_ERR_ARG, "struct_size %zu != sizeof(kda_rotary_args) %zu", a->struct_size,
         sizeof(kda_rotary_args));
  if (a->dtype != KDA_F32 && a->dtype != KDA_BF16 && a->dtype != KDA_F16)
    FAIL(KDA_ERR_DTYPE, "unknown dtype %d", a->dtype);
  const bool has_k = a->k != nullptr;
  if (a->total_tokens < 0) FAIL(KDA_ERR_SHAPE, "total_tokens must be >= 0");
  if (a->hq <= 0 || (has_k && a->hk <= 0)) FAIL(KDA_ERR_SHAPE, "head counts must be > 0");
  if (a->head_dim <= 0) FAIL(KDA_ERR_SHAPE, "head_dim must be > 0");
  if (a->head_dim % 8 != 0 || a->head_dim > MAX_DIM)
    FAIL(KDA_ERR_UNSUPPORTED, "head_dim must be a multiple of 8 and at most %d, got %d", MAX_DIM, a->head_dim);
  if (a->pairs < 1 || a->pairs > a->head_dim / 2)
    FAIL(KDA_ERR_SHAPE, "pairs must lie in [1, head_dim / 2], got %d", a->pairs);
  if (!isfinite(a->scale)) FAIL(KDA_ERR_SHAPE, "scale must be finite");
  const int64_t es = a->dtype == KDA_F32 ? 4 : 2, max_stride = (int64_t)1 << 24;
  RotaryLaunch L = {};
  const int64_t hk = has_k ? a->hk : 0;
  struct Side {
    const char* name;
    int64_t given, dense;
    int64_t* out;
    bool used;
  } sides[] = {{"q_stride", a->q_stride, (int64_t)a->hq * a->head_dim, &L.qs, true},
               {"k_stride", a->k_stride, hk * a->head_dim, &L.ks, has_k},
               {"q_out_stride", a->q_out_stride, (int64_t)a->hq * a->head_dim, &L.qos, true},
               {"k_out_stride", a->k_out_stride, hk * a->head_dim, &L.kos, has_k}};
  for (const Side& s : sides) {
    if (!s.used) continue;
    *s.out = s.given ? s.given : s.dense;
    if (*s.out < s.dense || *s.out > max_stride)
      FAIL(KDA_ERR_SHAPE, "%s %lld must be 0 or in [%lld, 2^24]", s.name, (long long)s.given, (long long)s.dense);
    if (*s.out * es % 16 != 0)
      FAIL(KDA_ERR_ARG, "%s %lld must keep rows 16-byte aligned", s.name, (long long)s.given);
  }
  if (a->total_tokens > (int64_t)INT32_MAX / ((a->hq + hk) * a->head_dim * es / 16))
    FAIL(KDA_ERR_UNSUPPORTED, "total_tokens * heads * head_dim above 2^31-1 16-byte pieces");
  // Tokens that share a workgroup: 32768 of 40 heads 127 us by four, 132 us one by one; 4096 the
  // same either way, 2048 13.0 and 9.8 us, 256 4.6 and 3.4 us.
  L.tb = a->total_tokens >= 4096 ? MAX_TB : 1;
  if ((a->total_tokens + L.tb - 1) / L.tb > MAX_GROUPS)
    FAIL(KDA_ERR_UNSUPPORTED, "total_tokens above 2^26 - 4");
  for (const void* p : {a->q, a->k, (const void*)a->q_out, (const void*)a->k_out})
    if (reinterpret_cast<uintptr_t>(p) & 15) FAIL(KDA_ERR_ARG, "tensor base pointers must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(a->positions) & 3 || reinterpret_cast<uintptr_t>(a->frequencies) & 7)
    FAIL(KDA_ERR_ARG, "positions and frequencies must be aligned to their elements");
  if (a->total_tokens == 0) return (kda_status)set_ok();
  if (!a->q || !a->q_out || (has_k && !a->k_out) || !a->positions || !a->frequencies)
    FAIL(KDA_ERR_ARG, "q, q_out, k_out (with k), positions and frequencies must be non-NULL");
  const RowSet q = {(uintptr_t)a->q, a->hq * a->head_dim * es, L.qs * es},
               k = {(uintptr_t)a->k, hk * a->head_dim * es, L.ks * es},
               qo = {(uintptr_t)a->q_out, q.row, L.qos * es}, ko = {(uintptr_t)a->k_out, k.row, L.kos * es};
  const bool q_here = q.at == qo.at && q.stride == qo.stride, k_here = has_k && k.at == ko.at && k.stride == ko.stride;
  const int64_t T = a->total_tokens;
  if ((!q_here && share(q, qo, T)) ||
      (has_k && ((!k_here && share(k, ko, T)) || share(q, ko, T) || share(k, qo, T) || share(qo, ko, T))))
    FAIL(KDA_ERR_ARG, "outputs must be their inputs or share no memory with them or one another");
  const RowSet lists[] = {{(uintptr_t)a->positions, 4 * T, 4 * T},
                          {(uintptr_t)a->frequencies, 8 * (int64_t)a->pairs, 8 * (int64_t)a->pairs}};
  for (const RowSet& s : lists)
    for (const RowSet& o : {qo, ko})
      if (o.at != 0 && s.at < o.at + (uintptr_t)((T - 1) * o.stride + o.row) && o.at < s.at + (uintptr_t)s.row)
        FAIL(KDA_ERR_ARG, "positions and frequencies must not lie among the outputs");
  const int V = (int)(16 / es);
  const bool inter = a->interleaved != 0, wide = (inter ? 2 * a->pairs : a->pairs) % V == 0;
  L.q = a->q; L.k = a->k; L.qo = a->q_out; L.ko = a->k_out;
  L.pos = a->positions; L.freq = a->frequencies;
  L.tokens = T;
  L.hq = a->hq; L.heads = a->hq + (int)hk; L.dim = a->head_dim; L.n = a->pairs;
  L.turns = !wide ? a->pairs : inter ? 2 * a->pairs / V : a->pairs / V;
  const int pass = q_here && (k_here || !has_k) ? 0 : (a->head_dim - 2 * a->pairs) / (wide ? V : 1);
  L.units = L.turns + pass;
  L.by_units = fast_div((uint32_t)L.units);
  L.by_heads = fast_div((uint32_t)L.heads);
  L.by_n = fast_div((uint32_t)L.n);
  L.scale = a->scale;
  L.sign = a->inverse ? -a->scale : a->scale;
  if (a->dtype == KDA_F32) rotary_go<float>(L, inter, wide, (hipStream_t)a->stream);
  else if (a->dtype == KDA_BF16) rotary_go<bf16>(L, inter, wide, (hipStream_t)a->stream);
  else rotary_go<_Float16>(L, inter, wide, (hipStream_t)a->stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) FAIL(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  return (kda_status)set_ok();
}
