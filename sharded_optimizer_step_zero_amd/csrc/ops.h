// ops.h -- what the model operators' kernels share: reading and writing rows of
// any element type eight elements at a time, the 8-bit form, and argument checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>
#include <type_traits>

#include "../../include/zeroshard.h"
#include "../../include/zeroshard_ops.h"
#include "abi_internal.h"

namespace zs {
namespace ops {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

template <int DT>
struct Elem;
template <>
struct Elem<ZS_F32> {
  using type = float;
  using vec = f32x8;
};
template <>
struct Elem<ZS_BF16> {
  using type = __bf16;
  using vec = bf16x8;
};
template <>
struct Elem<ZS_F16> {
  using type = _Float16;
  using vec = f16x8;
};
template <int DT>
using elem_t = typename Elem<DT>::type;

// Wide accesses at any element's address: global memory is read and written
// unaligned, so a row may start anywhere.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

// NT: the data passes once and does not fit the caches; it is kept out of them.
template <bool NT>
__device__ __forceinline__ u32x4 ld16(const void* p) {
  if (NT) return __builtin_nontemporal_load((const u32x4_any*)p);
  return *(const u32x4_any*)p;
}
template <bool NT>
__device__ __forceinline__ void st16(void* p, u32x4 x) {
  if (NT)
    __builtin_nontemporal_store(x, (u32x4_any*)p);
  else
    *(u32x4_any*)p = x;
}

// Eight elements of a row as they lie in memory: a lane's chunk.
template <int DT>
struct Chunk {
  static constexpr int kWords = DT == ZS_F32 ? 2 : 1;
  u32x4 w[kWords];
};
// The chunk at p, n elements of which exist (the rest are 0).
template <int DT, bool NT = false>
__device__ __forceinline__ Chunk<DT> load_chunk(const elem_t<DT>* p, int64_t n) {
  Chunk<DT> r;
  if (n >= 8) {
#pragma unroll
    for (int i = 0; i < Chunk<DT>::kWords; i++) r.w[i] = ld16<NT>((const u32x4_any*)p + i);
    return r;
  }
  elem_t<DT> e[8];
#pragma unroll
  for (int i = 0; i < 8; i++) e[i] = i < n ? p[i] : (elem_t<DT>)0.0f;
  __builtin_memcpy(&r, e, sizeof(r));
  return r;
}
template <int DT>
__device__ __forceinline__ f32x8 widen(Chunk<DT> c) {
  return __builtin_convertvector(__builtin_bit_cast(typename Elem<DT>::vec, c), f32x8);
}
// The chunk of a row from element c on without a branch, so that loads under way are
// not waited for where a row ends inside a wave: where the row ends before the
// chunk does, its last eight elements, which take8() moves into place.  Rows
// narrower than that are read element by element.
template <int DT, bool NT = false>
__device__ __forceinline__ Chunk<DT> load_row(const elem_t<DT>* row, int64_t c, int64_t width) {
  if (width < 8) return load_chunk<DT>(row + c, width - c);
  const elem_t<DT>* p = row + (c + 8 <= width ? c : width - 8);
  Chunk<DT> r;
#pragma unroll
  for (int i = 0; i < Chunk<DT>::kWords; i++) r.w[i] = ld16<NT>((const u32x4_any*)p + i);
  return r;
}
// load_row's chunk as fp32, n elements of it (of a row of `width`) in place and
// zeros behind them; n <= 0: zeros.
template <int DT>
__device__ __forceinline__ f32x8 take8(Chunk<DT> x, int64_t n, int64_t width) {
  const f32x8 v = widen<DT>(x);
  f32x8 r = {};
  if (n >= 8 || (width < 8 && n > 0)) return v;
#pragma unroll
  for (int k = 1; k < 8; k++)
    if (n == k) {
#pragma unroll
      for (int i = 0; i < k; i++) r[i] = v[i + 8 - k];
    }
  return r;
}
// Eight elements as fp32.
template <int DT, bool NT = false>
__device__ __forceinline__ f32x8 load8(const elem_t<DT>* p, int64_t n) {
  return widen<DT>(load_chunk<DT, NT>(p, n));
}

// Rounds to the element type (nearest, ties to even) and stores.
template <int DT, bool NT = false>
__device__ __forceinline__ void store8(elem_t<DT>* p, int64_t n, f32x8 x) {
  const typename Elem<DT>::vec v = __builtin_convertvector(x, typename Elem<DT>::vec);
  if (n >= 8) {
    const Chunk<DT> c = __builtin_bit_cast(Chunk<DT>, v);
#pragma unroll
    for (int i = 0; i < Chunk<DT>::kWords; i++) st16<NT>((u32x4_any*)p + i, c.w[i]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; i++)
    if (i < n) p[i] = v[i];
}

// ---------------------------------------------------------------- 8-bit form

// The scale byte of a group with this largest magnitude.  1.75 * 2^top is the
// format's largest value: a mantissa above .75 goes to the next power of two.
template <int CODE>
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  constexpr int top = CODE == ZS_E4M3 ? 8 : 15;
  const uint32_t b = __float_as_uint(amax);
  if (b >= 0x7f800000u) return 255u;
  const int e = (int)((b + 0x1fffffu) >> 23) - top;  // biased by 127
  return (uint32_t)(e < 0 ? 0 : e);
}
// 2^-e of a scale byte that is not 255 (byte 0: 2^127), and 2^e (255: NaN).
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float scale_value(uint32_t byte) {
  if (byte == 255u) return __uint_as_float(0x7fc00000u);
  return byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u);
}

template <int CODE>
__device__ __forceinline__ u32x2 encode8(f32x8 x) {
  u32x2 r;
#pragma unroll
  for (int h = 0; h < 2; h++) {
    int w = 0;
    if (CODE == ZS_E4M3) {
      w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h], x[4 * h + 1], w, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h + 2], x[4 * h + 3], w, true);
    } else {
      w = __builtin_amdgcn_cvt_pk_bf8_f32(x[4 * h], x[4 * h + 1], w, false);
      w = __builtin_amdgcn_cvt_pk_bf8_f32(x[4 * h + 2], x[4 * h + 3], w, true);
    }
    r[h] = (uint32_t)w;
  }
  return r;
}
template <int CODE>
__device__ __forceinline__ f32x8 decode8(u32x2 w) {
  f32x8 r;
#pragma unroll
  for (int h = 0; h < 2; h++) {
    f32x2 a, b;
    if (CODE == ZS_E4M3) {
      a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
      b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
    } else {
      a = __builtin_amdgcn_cvt_pk_f32_bf8((int)w[h], false);
      b = __builtin_amdgcn_cvt_pk_f32_bf8((int)w[h], true);
    }
    r[4 * h] = a[0];
    r[4 * h + 1] = a[1];
    r[4 * h + 2] = b[0];
    r[4 * h + 3] = b[1];
  }
  return r;
}

// Eight codes at p, n of them exist.
template <bool NT = false>
__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int64_t n) {
  if (n >= 8) return NT ? __builtin_nontemporal_load((const u32x2_any*)p) : *(const u32x2_any*)p;
  u32x2 r = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; i++)
    if (i < n) r[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
  return r;
}
template <bool NT = false>
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t n, u32x2 w) {
  if (n >= 8) {
    if (NT)
      __builtin_nontemporal_store(w, (u32x2_any*)p);
    else
      *(u32x2_any*)p = w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; i++)
    if (i < n) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
}

// |x| as bits: integer order is the order of magnitudes, with NaN above
// infinity, so a group's maximum also tells that it holds one.
__device__ __forceinline__ uint32_t amax_bits(f32x8 x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7fffffffu;
    m = b > m ? b : m;
  }
  return m;
}
// The maximum over the 4, 8 or 16 neighbouring lanes (8 elements each) of a group.
__device__ __forceinline__ float group_amax(f32x8 x, int lanes) {
  uint32_t m = amax_bits(x);
  for (int d = 1; d < lanes; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)m, d, 64);
    m = o > m ? o : m;
  }
  return __uint_as_float(m);
}
// The codes of the lane's eight elements and their group's scale byte, given the
// group's largest magnitude.
template <int CODE>
__device__ __forceinline__ u32x2 quantise8(f32x8 x, float amax, uint32_t* byte) {
  const uint32_t b = scale_byte<CODE>(amax);
  *byte = b;
  const float inv = scale_inverse(b == 255u ? 127u : b);
  f32x8 s;
#pragma unroll
  for (int i = 0; i < 8; i++) s[i] = x[i] * inv;
  u32x2 w = encode8<CODE>(s);
  if (b == 255u) w = u32x2{0, 0};
  return w;
}

// ---------------------------------------------------------------- host side

inline int fail(const char* who, const char* what) {
  return einval((std::string(who) + ": " + what).c_str());
}
inline int elem_bytes(int32_t dtype) { return dtype == ZS_F32 ? 4 : 2; }
inline bool good_dtype(int32_t d) { return d >= ZS_F32 && d <= ZS_F16; }
inline bool good_group(int32_t g) { return g == 32 || g == 64 || g == 128; }
inline bool al(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }
// Rows that can be read 16 bytes at a time.
inline bool wide(const void* p, int64_t stride, int32_t dtype) {
  return al(p, 16) && (stride * elem_bytes(dtype)) % 16 == 0;
}
// Whether a call's arrays together pass the last-level cache (256 MB), so that
// what it writes is gone from there before it is read again.  Streamed accesses gain 3
// to 7% there in 16-bit types.  A chunk of fp32 takes two accesses, each half of every
// line, and loses 10% (norm, 16384 x 8192: 432 against 478 us): its callers do without.
inline bool streams(int64_t bytes) { return bytes >= (256ll << 20); }
inline int launched(const char* who) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? ZS_OK : ehip(who, e);
}
inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Calls f with the type as a constant.
template <typename F>
inline void with_dtype(int32_t dtype, F f) {
  if (dtype == ZS_F32)
    f(std::integral_constant<int, ZS_F32>());
  else if (dtype == ZS_BF16)
    f(std::integral_constant<int, ZS_BF16>());
  else
    f(std::integral_constant<int, ZS_F16>());
}
template <typename F>
inline void with_bool(bool b, F f) {
  if (b)
    f(std::integral_constant<bool, true>());
  else
    f(std::integral_constant<bool, false>());
}
template <typename F>
inline void with_code(int32_t code, F f) {
  if (code == ZS_E4M3)
    f(std::integral_constant<int, ZS_E4M3>());
  else
    f(std::integral_constant<int, ZS_E5M2>());
}

}  // namespace ops
}  // namespace zs
