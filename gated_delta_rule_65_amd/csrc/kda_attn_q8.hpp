// The paged cache in 8 bits: launch descriptors and what its kernels share (gfx950).
//
// A value is its block's scale, a power of two, times a code (e4m3 or a signed byte).
// Either has at most 8 significant bits, so it is a bf16 number, and the widening
// conversions below are exact.
#pragma once
#include "kda_attn.hpp"

namespace kda {

constexpr int E4M3 = 0, INT8 = 1;  // kda_code

// What addresses the cache in 8 bits beside AttnLaunch's pools.
struct Scales {
  const float *k, *v;  // [num_pages, hkv, per_page]
  FastDiv block;       // by the positions of a scale
  int per_page;
};
struct AttnQ8Launch : AttnLaunch {  // k_page and v_page in bytes, as there
  Scales scales;
  int code;
};
hipError_t launch_attn_q8_rows(const AttnQ8Launch& L);
hipError_t launch_attn_q8_tiles(const AttnQ8Launch& L);

// New rows into the cache, or cached rows out of it.
struct CacheQ8Launch {
  const void *k, *v;       // rows in (append)
  void *ko, *vo;           // rows out (read)
  void *kc, *vc;           // codes
  float *ks, *vs;          // [num_pages, hkv, per_page]
  const int32_t *table, *cu, *seq;
  int64_t k_stride, v_stride;  // bytes between tokens of k and v
  int64_t k_page, v_page;      // bytes between pages
  int64_t table_stride;
  int64_t capacity;            // max_pages * page size
  int dtype, code, n, total, hkv, dim, num_pages, max_pages, per_page;
  FastDiv page, block, hdiv;   // by the page size, the positions of a scale, hkv
  void* stream;
};
hipError_t launch_append_q8(const CacheQ8Launch& L);
hipError_t launch_read_q8(const CacheQ8Launch& L);

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2v_t __attribute__((ext_vector_type(2)));

// A block's scale as it was loaded: the power of two of its exponent, sign and lower bits dropped.  e4m3's
// conversion reads scales so by itself; everything else that takes one goes through here, so that
// a scale that is no power of two stands for the same values in every operator.
__device__ __forceinline__ float pow2_scale(float s) {
  return __uint_as_float(__float_as_uint(s) & 0x7f800000u);
}

// The four codes of a word.
template <int CODE> struct Code;
template <> struct Code<E4M3> {
  // as fp32, unscaled
  static __device__ __forceinline__ void widen(uint32_t w, float (&x)[4]) {
    const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1];
  }
  // as 16-bit values times s (the conversion takes s by its exponent)
  static __device__ __forceinline__ u32x2v_t widen16(bf16, uint32_t w, float s) {
    return u32x2v_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true))};
  }
  static __device__ __forceinline__ u32x2v_t widen16(_Float16, uint32_t w, float s) {
    return u32x2v_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s, false)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s, true))};
  }
  // The codes of four values already divided by their scale: to nearest, ties to even.
  // What is no finite number becomes NaN.
  static __device__ __forceinline__ uint32_t encode(const float (&x)[4]) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w, true);
  }
  // The least power of two s >= 2^-126 with top <= 448 s, for top >= 0: 448 is 1.75 * 2^8.
  static __device__ __forceinline__ float least_scale(float top) {
    const uint32_t u = __float_as_uint(top);
    const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u);
    return __uint_as_float((uint32_t)max(e, 1) << 23);
  }
};
template <> struct Code<INT8> {
  static __device__ __forceinline__ void widen(uint32_t w, float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(w >> (8 * i));
  }
  // (A known device.)  The low byte of an fp16 number of 2^10 is its integer part: put there, the unsigned byte b + 128
  // makes 1152 + b, and (1152 + b) s - 1152 s is one instruction that takes its fp16 operand
  // as it is.  Every step is exact (1152 s is a number: values lie below 2^99).  By conversions
  // of bytes to fp32 it was 11 instructions for four codes in place of 9: 2048 tokens on 131072
  // keys 4.13 ms, now 3.94; 24 ragged prompts 895 us, now 881.  s is a power of two (pow2_scale).
  template <typename E> static __device__ __forceinline__ u32x2v_t widen16(E, uint32_t w, float s) {
    const uint32_t u = w ^ 0x80808080u;
    const f16x2_t a = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u));
    const f16x2_t b = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u));
    const float z = -1152.0f * s;
    const float x0 = fmaf((float)a[0], s, z), x1 = fmaf((float)a[1], s, z);
    const float x2 = fmaf((float)b[0], s, z), x3 = fmaf((float)b[1], s, z);
    if constexpr (std::is_same_v<E, bf16>) {
      return u32x2v_t{__builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)x0, (__bf16)x1}),
                      __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)x2, (__bf16)x3})};
    } else {
      return u32x2v_t{__builtin_bit_cast(uint32_t, f16x2_t{(_Float16)x0, (_Float16)x1}),
                      __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)x2, (_Float16)x3})};
    }
  }
  // To nearest, ties to even; NaN becomes 0 and infinities +-127.
  static __device__ __forceinline__ uint32_t encode(const float (&x)[4]) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float y = x[i] == x[i] ? fminf(fmaxf(x[i], -127.0f), 127.0f) : 0.0f;
      w |= ((uint32_t)(int)__builtin_rintf(y) & 0xffu) << (8 * i);
    }
    return w;
  }
  // 127 is 1.984375 * 2^6.
  static __device__ __forceinline__ float least_scale(float top) {
    const uint32_t u = __float_as_uint(top);
    const int e = (int)(u >> 23) - 6 + ((u & 0x7fffffu) > 0x7e0000u);
    return __uint_as_float((uint32_t)max(e, 1) << 23);
  }
};

// 1 / s of a power of two between 2^-126 and 2^126.
__device__ __forceinline__ float inverse_scale(float s) {
  return __uint_as_float((254u << 23) - __float_as_uint(s));
}

// A request's rows: the first, their number, and its length.
struct Rows {
  int req, start, len, seq;
};
// The last request whose first item (by `first` of its index and first row, which grows with the index)
// is at most `item`; all lanes of a wave ask together.  Up to 256 requests are looked through
// in one round trip to memory, offsets and lengths at once; more take one per factor of 64.
template <typename F>
__device__ __forceinline__ Rows find_rows(const int32_t* cu, const int32_t* seq, int n, int total, int item,
                                          int lane, F first) {
  Rows r;
  auto clamp = [&](int c) { return min(max(c, 0), total); };
  if (n <= 256) {
    constexpr int M = 4;
    int c[M], s[M];
    const int last = clamp(cu[n]);
#pragma unroll
    for (int j = 0; j < M; ++j) {
      c[j] = s[j] = 0;
      if (64 * j < n) {
        const int i = min(64 * j + lane, n - 1);
        c[j] = clamp(cu[i]);
        s[j] = seq[i];
      }
    }
    r.req = -1;
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int i = 64 * j + lane;
      r.req += __popcll(__ballot(i == 0 || (i < n && first(i, c[j]) <= item)));
    }
    auto at = [&](const int (&v)[M], int i) {
      const int x = i < 64 ? v[0] : i < 128 ? v[1] : i < 192 ? v[2] : v[3];
      return __builtin_amdgcn_readlane(x, i & 63);
    };
    r.start = at(c, r.req);
    r.len = max(r.req + 1 < n ? at(c, r.req + 1) : last, r.start) - r.start;
    r.seq = max(at(s, r.req), 0);
    return r;
  }
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) / 64;
    const int i = lo + lane * step;
    const bool in = lane == 0 || (i < hi && first(i, clamp(cu[i])) <= item);
    const int k = __popcll(__ballot(in)) - 1;
    lo += k * step;
    hi = min(hi, lo + step);
  }
  r.req = lo;
  r.start = clamp(cu[lo]);
  r.len = max(clamp(cu[lo + 1]), r.start) - r.start;
  r.seq = max(seq[lo], 0);
  return r;
}

}  // namespace kda
