// mx4.hip -- matrices in 4 bits with a scale for each 32 neighbours, and their product.
//
// Packing: a group's scale is the least power of two that brings it within 6, its codes the
// elements over that scale rounded to {0, 1/2, 1, 3/2, 2, 3, 4, 6}, ties to even: 17 bytes for 32
// elements.  Bound by HBM.  Along rows a lane has 8 elements and a group's maximum is one over
// 4 neighbouring lanes.  Along columns (the transpose's rows) a lane has 32 rows of four columns in
// registers, so that a column's group is its own; with both wanted a row's group is eight
// lanes', and the matrix is read once.  16-bit elements are compared and rounded as they are, two
// at a time.  8192 x 22016 bf16, which passes the last-level cache, both ways 125 us (4.4 TB/s), along
// rows 87 (5.2); 22016 x 4096 69 and 43 from HBM, 57 and 38 where the cache holds it from before.
// (A tile of 128 x 128 turned in LDS, its 16-byte and single-byte pieces written apart: 150.)
//
// The product: out[t][n] = sum_k x[t][k] w[n][k] of the values codes * scales, on 16x16x128
// matrix instructions that take the scales themselves (4-bit in, fp32 sums), one rounding at
// the end.  A lane of an instruction has one row's group of 32: 16 bytes of codes and a
// byte of a register that holds the scales of four instructions; the scales lie in memory in
// just that order (scale4_at), so that they go the codes' way with no rearrangement.
//
// All tiles take 256 k a step, two steps in LDS, which global memory is read straight into: a row
// has 128 bytes there, a cache line of memory (64-byte pieces of lines have twice the requests,
// which the L2 answers no faster than one a channel and cycle: 8192 x 4096 x 22016 took 430 us).  A
// row's chunk c of 16 bytes sits at c ^ (row & 7): no bank conflicts.  Rows past the edge and groups
// past the end read as zeros by the buffer loads' bounds check.
//
// Large products: 256 x 256, four waves of 128 x 128 whose sums fill the accumulation registers
// (eight waves of 128 x 64: 460 us).  A half step's fragments are read while the half before
// is multiplied; between the halves is the step's one barrier, where the next step's codes,
// under way for a step and a half, have landed and this one's place is free.  A workgroup goes
// on from tile to tile: the next one's first loads are under way before the last one's
// products end, and its rows leave through LDS in pieces of 256 bytes (32-byte pieces straight
// from the registers: 402 us; 64-byte ones: 368; these 357, and 330 streamed).  Smaller products take
// 128 x 128 or 128 x 64 tiles, two or three workgroups a compute unit.
//
// Few tokens: the weight is what is read, each of its rows by one workgroup, whose waves share
// k out between them and add their sums in LDS: 16 x 4096 x 22016 in a graph 13.6 us (3.5 TB/s, weights
// from HBM; a pass of 48 MB has about 3 us of start and end, a wave has one span of this width and
// nothing under way behind it, and the tokens' codes come again for every 32 features: one token
// 11.5 us).
//
// Measured, bf16 out: 8192 x 22016 x 4096 (tokens x width x features) 285 us, 5.2 PFLOP/s; 22016 x
// 8192 x 4096 327 us; 8192 x 4096 x 22016, sixteen steps a tile and 360 MB to write, 330 us, 4.5
// PFLOP/s.  What bounds them is the card's power (on zeros, at a higher clock, the first takes 232 us, 6.4
// PFLOP/s) and LDS: a half step's 1024 cycles of matrix instructions come with 64 KB of fragments read
// and 32 KB of codes written there, at 128 bytes a cycle three quarters of them; the matrix cores are
// busy for 55% of the cycles.
#include <algorithm>

#include "ops.h"

namespace zs {
namespace ops {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
#define ZS_LDS __attribute__((address_space(3)))

constexpr int64_t kMaxSide = 1ll << 24;   // rows of an operand
constexpr int64_t kMaxWidth = 1ll << 20;
constexpr int kRsrcWord3 = 0x00020000;  // raw 32-bit buffer, gfx9 family
constexpr int64_t groups_of(int64_t width) { return (width + 31) / 32; }
constexpr int64_t spans_of(int64_t width) { return (width + 511) / 512; }

// ---------------------------------------------------------------- packing

// Codes and scale byte of a lane's eight elements, given their group's largest magnitude.
__device__ __forceinline__ uint32_t quantise4(f32x8 x, float amax, uint32_t* byte) {
  const uint32_t b = scale_byte<ZS_E2M1>(amax);
  *byte = b;
  const float inv = scale_inverse(b == 255u ? 127u : b);
  f32x8 s;
#pragma unroll
  for (int i = 0; i < 8; i++) s[i] = x[i] * inv;
  const uint32_t w = encode4(s, 1.0f);
  return b == 255u ? 0u : w;
}

// A chunk of eight a thread, a row's chunks up to whole spans of 512.
template <int DT, bool NT>
__global__ __launch_bounds__(256) void pack_rows_kernel(const elem_t<DT>* __restrict__ x,
                                                        int64_t x_stride,
                                                        uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales, int64_t rows,
                                                        int64_t width, int64_t groups,
                                                        uint32_t blocks_per_row) {
  const int64_t row = (int64_t)(blockIdx.x / blocks_per_row) * 4 + (threadIdx.x >> 6);
  const int64_t chunk = (int64_t)(blockIdx.x % blocks_per_row) * 64 + (threadIdx.x & 63);
  if (row >= rows) return;  // whole waves
  const int64_t c = chunk * 8, group = chunk >> 2;
  const f32x8 v = c < width ? load8<DT, NT>(x + row * x_stride + c, width - c) : f32x8{};
  uint32_t byte;
  const uint32_t w = quantise4(v, group_amax(v, 4), &byte);
  if (group < groups) *(uint32_t*)(codes + row * groups * 16 + chunk * 4) = w;
  if ((chunk & 3) == 0) scales[scale4_at(row, group, rows)] = (uint8_t)(group < groups ? byte : 127u);
}

// The largest of a group's eight lanes (four elements each), in each half of a word by itself.
template <typename MAX>
__device__ __forceinline__ uint32_t eight_lanes(uint32_t m, MAX max) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xb1, 0xf, 0xf, true));   // lane ^ 1
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4e, 0xf, 0xf, true));   // lane ^ 2
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xf, 0xf, true));  // 7 - lane
}

// A group's scale byte, and the scale for the instruction that encodes: it takes the exponent
// field only, which is 0 for 2^-127 too.
__device__ __forceinline__ uint32_t byte4(float amax, float* scale) {
  const uint32_t b = scale_byte<ZS_E2M1>(amax);
  *scale = __uint_as_float(b << 23);
  return b;
}

// From so many blocks of 256 x 256 on; below, 64 x 256, so that the card has work.  us with large and
// with small blocks, bf16 from HBM: 8192 x 4096 (512) 31 and 24, 22016 x 4096 (1376) 69 and 72, 8192
// x 22016 (2752) 126 and 178.
constexpr int64_t kLargeBlocks = 1024;

// WAVES * 32 rows x 256 columns: a lane has 32 rows of four columns, so that a group along columns
// is one lane's and a group along rows eight lanes'.  ROWS: both, else along columns only.
template <int DT, bool ROWS, int WAVES>
__global__ __launch_bounds__(WAVES * 64, DT == ZS_F32 ? 2 : 4) void pack_both_kernel(
    const elem_t<DT>* __restrict__ x, int64_t x_stride, uint8_t* __restrict__ codes,
    uint8_t* __restrict__ scales, uint8_t* __restrict__ codes_t, uint8_t* __restrict__ scales_t,
    int64_t rows, int64_t width, uint32_t tiles_down) {
  __shared__ __attribute__((aligned(16))) u32x4 turned[256 * WAVES];
  __shared__ uint8_t bytes[256 * WAVES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));  // rows are scalars
  const int64_t r0 = (int64_t)(blockIdx.x % tiles_down) * (WAVES * 32), row0 = r0 + wave * 32;
  const int64_t c0 = (int64_t)(blockIdx.x / tiles_down) * 256;
  const int c = lane * 4;  // in the block
  const int64_t groups = groups_of(width), groups_t = groups_of(rows);
  constexpr bool kWide = DT == ZS_F32;
  constexpr int kWords = kWide ? 4 : 2;
  uint32_t w[32][kWords];
  const elem_t<DT>* p = x + row0 * x_stride + c0;
  const int64_t there = width - c0;  // columns that exist
  if (row0 + 32 <= rows && there >= 256) {
#pragma unroll
    for (int i = 0; i < 32; i++) {
      if constexpr (kWide)
        __builtin_memcpy(w[i], (const u32x4_any*)(p + i * x_stride + c), 16);
      else
        __builtin_memcpy(w[i], (const u32x2_any*)(p + i * x_stride + c), 8);
    }
  } else if (there >= 4) {
    // Without a branch in a lane: where the row ends before the lane's elements do, its last
    // four, which move into place.
    const int from = c + 4 <= there ? c : (int)there - 4, by = c - from;
#pragma unroll
    for (int i = 0; i < 32; i++) {
      const elem_t<DT>* q = x + (row0 + i < rows ? row0 + i : rows - 1) * x_stride + c0;
      if constexpr (kWide)
        __builtin_memcpy(w[i], (const u32x4_any*)(q + from), 16);
      else
        __builtin_memcpy(w[i], (const u32x2_any*)(q + from), 8);
    }
#pragma unroll
    for (int i = 0; i < 32; i++) {
      const bool none = row0 + i >= rows;
      if constexpr (kWide) {
#pragma unroll
        for (int k = 0; k < 4; k++) w[i][k] = by & 1 ? (k < 3 ? w[i][k + 1 & 3] : 0u) : w[i][k];
#pragma unroll
        for (int k = 0; k < 4; k++) w[i][k] = by & 2 ? (k < 2 ? w[i][k + 2 & 3] : 0u) : w[i][k];
#pragma unroll
        for (int k = 0; k < 4; k++) w[i][k] = none || by >= 4 ? 0u : w[i][k];
      } else {
        uint64_t v;
        __builtin_memcpy(&v, w[i], 8);
        v = none || by >= 4 ? 0ull : v >> (by * 16 & 63);
        __builtin_memcpy(w[i], &v, 8);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; i++) {
      elem_t<DT> e[4];
#pragma unroll
      for (int k = 0; k < 4; k++)
        e[k] = row0 + i < rows && c + k < there ? p[i * x_stride + c + k] : (elem_t<DT>)0.0f;
      __builtin_memcpy(w[i], e, sizeof(w[i]));
    }
  }
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  auto max16 = [](uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
  };
  auto max32 = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  // a magnitude's bits as fp32 (16-bit types: in the low half)
  auto value = [](uint32_t bits) {
    if constexpr (DT == ZS_F32) return __uint_as_float(bits);
    if constexpr (DT == ZS_BF16) return __uint_as_float(bits << 16);
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  };
  // two elements' codes into byte AT of a word; 16-bit types: both in `a`
  auto encode = [](auto AT, uint32_t old, uint32_t a, uint32_t b, float scale) {
    constexpr int at = decltype(AT)::value;
    typedef elem_t<DT> pair_t __attribute__((ext_vector_type(2)));
    if constexpr (DT == ZS_F32)
      return (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32((int)old, __uint_as_float(a), __uint_as_float(b), scale, at);
    else if constexpr (DT == ZS_BF16)
      return (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_bf16((int)old, __builtin_bit_cast(pair_t, a), scale, at);
    else
      return (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f16((int)old, __builtin_bit_cast(pair_t, a), scale, at);
  };
  std::integral_constant<int, 0> b0;
  std::integral_constant<int, 1> b1;
  std::integral_constant<int, 2> b2;
  std::integral_constant<int, 3> b3;

  uint32_t columns[kWords] = {};  // the columns' largest magnitudes, as the elements lie
  const int64_t group0 = c0 / 32;
  const bool exists = group0 + (lane >> 3) < groups;
  uint32_t eighth = 0;  // of eight rows, the scale byte of the one that this lane writes
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    uint32_t m[2];
#pragma unroll
    for (int q = 0; q < 2; q++) {
      uint32_t s[kWords];
#pragma unroll
      for (int k = 0; k < kWords; k++) {
        s[k] = w[i + q][k] & (kWide ? 0x7fffffffu : 0x7fff7fffu);
        columns[k] = kWide ? max32(columns[k], s[k]) : max16(columns[k], s[k]);
      }
      if constexpr (kWide)
        m[q] = max32(max32(s[0], s[1]), max32(s[2], s[3]));
      else
        m[q] = max16(s[0], s[1]);
    }
    if (ROWS) {
      if constexpr (kWide) {
        m[0] = eight_lanes(m[0], max32);
        m[1] = eight_lanes(m[1], max32);
      } else {  // two rows in a word
        uint32_t both = max16(__builtin_amdgcn_perm(m[1], m[0], 0x05040100), __builtin_amdgcn_perm(m[1], m[0], 0x07060302));
        both = eight_lanes(both, max16);
        m[0] = both & 0xffffu;
        m[1] = both >> 16;
      }
#pragma unroll
      for (int q = 0; q < 2; q++) {
        float scale;
        const uint32_t byte = byte4(value(m[q]), &scale);
        uint32_t code;
        if constexpr (kWide)
          code = encode(b1, encode(b0, 0u, w[i + q][0], w[i + q][1], scale), w[i + q][2], w[i + q][3], scale);
        else
          code = encode(b1, encode(b0, 0u, w[i + q][0], 0u, scale), w[i + q][1], 0u, scale);
        if (byte == 255u) code = 0;
        if ((lane & 7) == ((i + q) & 7)) eighth = byte;
        if (row0 + i + q < rows && exists)
          *(uint16_t*)(codes + (row0 + i + q) * groups * 16 + c0 / 2 + lane * 2) = (uint16_t)code;
      }
      if ((i & 7) == 6) {
        const int64_t row = row0 + i - 6 + (lane & 7);
        if (row < rows) scales[scale4_at(row, group0 + (lane >> 3), rows)] = (uint8_t)(exists ? eighth : 127u);
      }
    }
  }
  // The columns: 32 rows' codes are 16 bytes, which go through LDS so that a column's groups are
  // written together.  A column's place for a wave is turned by its lane, so that eight
  // neighbouring lanes meet different banks.
#pragma unroll
  for (int k = 0; k < 4; k++) {
    float scale;
    const uint32_t bits = kWide ? columns[k] : (k & 1 ? columns[k >> 1] >> 16 : columns[k >> 1] & 0xffffu);
    const uint32_t byte = byte4(value(bits), &scale);
    u32x4 word;
#pragma unroll
    for (int q = 0; q < 4; q++) {
      uint32_t code = 0;
      auto two = [&](auto AT) {
        const int i = q * 8 + decltype(AT)::value * 2;
        if constexpr (kWide)
          code = encode(AT, code, w[i][k], w[i + 1][k], scale);
        else
          code = encode(AT, code, __builtin_amdgcn_perm(w[i + 1][k >> 1], w[i][k >> 1], k & 1 ? 0x07060302 : 0x05040100), 0u, scale);
      };
      two(b0);
      two(b1);
      two(b2);
      two(b3);
      word[q] = byte == 255u ? 0u : code;
    }
    const int col = lane * 4 + k;
    turned[col * WAVES + (wave ^ (lane & (WAVES - 1)))] = word;
    bytes[col * WAVES + wave] = (uint8_t)byte;
  }
  __syncthreads();
  const int64_t g0 = r0 / 32;
#pragma unroll
  for (int n = 0; n < 4; n++) {
    const int at = threadIdx.x + n * WAVES * 64, col = at / WAVES, g = at % WAVES;
    if (c0 + col < width && g0 + g < groups_t)
      *(u32x4*)(codes_t + ((c0 + col) * groups_t + g0 + g) * 16) = turned[col * WAVES + (g ^ (col >> 2 & (WAVES - 1)))];
  }
  // scale bytes: a wave's groups g and g + 4 are neighbours
  if constexpr (WAVES == 8) {
#pragma unroll
    for (int n = 0; n < 2; n++) {
      const int at = threadIdx.x + n * 512, col = at / 4, g = at % 4;
      if (c0 + col >= width) continue;
      const uint32_t lo = g0 + g < groups_t ? bytes[col * 8 + g] : 127u;
      const uint32_t hi = g0 + g + 4 < groups_t ? bytes[col * 8 + g + 4] : 127u;
      *(uint16_t*)(scales_t + scale4_at(c0 + col, g0 + g, width)) = (uint16_t)(lo | hi << 8);
    }
  } else {
#pragma unroll
    for (int n = 0; n < 4; n++) {
      const int at = threadIdx.x + n * WAVES * 64, col = at / WAVES, g = at % WAVES;
      if (c0 + col < width)
        scales_t[scale4_at(c0 + col, g0 + g, width)] = g0 + g < groups_t ? bytes[at] : (uint8_t)127;
    }
  }
}

template <int DT, bool NT>
__global__ __launch_bounds__(256) void unpack_kernel(const uint8_t* __restrict__ codes,
                                                     const uint8_t* __restrict__ scales,
                                                     elem_t<DT>* __restrict__ x, int64_t x_stride,
                                                     int64_t rows, int64_t width, int64_t groups,
                                                     uint32_t blocks_per_row) {
  const int64_t row = (int64_t)(blockIdx.x / blocks_per_row) * 4 + (threadIdx.x >> 6);
  const int64_t chunk = (int64_t)(blockIdx.x % blocks_per_row) * 64 + (threadIdx.x & 63);
  const int64_t c = chunk * 8;
  if (row >= rows || c >= width) return;
  const uint32_t w = *(const uint32_t*)(codes + row * groups * 16 + chunk * 4);
  const float scale = scale_value(scales[scale4_at(row, chunk >> 2, rows)]);
  store8<DT, NT>(x + row * x_stride + c, width - c, decode4(w, 1.0f) * scale);
}

// ---------------------------------------------------------------- product

constexpr int kBig = 256;  // a large tile's side

struct Mx4Args {
  const uint8_t *a, *b;    // codes of w (features) and x (tokens)
  const uint8_t *as, *bs;  // scales
  int64_t m, n;            // features, tokens
  int32_t groups;          // of k
  int32_t tiles_m, tiles_n;
  void* c;
  int64_t ldc;
  int32_t streaming;       // the output passes the last-level cache
};

template <int J>
__device__ __forceinline__ f32x4 mfma4(i32x4 a, i32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  const i32x8 wa = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 wb = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, wb, c, 4, 4, J, (int)sa, J, (int)sb);
}

// Four neighbouring features of a token, `left` of which exist.
template <int DT>
__device__ __forceinline__ void store4(elem_t<DT>* p, int64_t left, f32x4 x) {
  typedef elem_t<DT> v4 __attribute__((ext_vector_type(4)));
  const v4 v = __builtin_convertvector(x, v4);
  if (left >= 4) {
    if constexpr (DT == ZS_F32)
      *(u32x4_any*)p = __builtin_bit_cast(u32x4, v);
    else
      *(u32x2_any*)p = __builtin_bit_cast(u32x2, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; i++)
    if (i < left) p[i] = v[i];
}

// The tile of a workgroup.  Workgroups go round the 8 dies: each die takes a contiguous part of
// the tiles, which run down a band of 8 tiles of tokens, so that the tiles at work on
// a die share their rows in its L2.
__device__ __forceinline__ void tile_of(const Mx4Args& g, int32_t* tm, int32_t* tn) {
  const uint32_t total = gridDim.x, die = blockIdx.x & 7, per = total >> 3, extra = total & 7;
  const uint32_t id = die * per + (die < extra ? die : extra) + (blockIdx.x >> 3);
  const uint32_t band = id / ((uint32_t)g.tiles_m * 8);
  const uint32_t in = id - band * (uint32_t)g.tiles_m * 8;
  const uint32_t wide = (uint32_t)g.tiles_n - band * 8 < 8 ? (uint32_t)g.tiles_n - band * 8 : 8;
  *tm = (int32_t)(in / wide);
  *tn = (int32_t)(band * 8 + in % wide);
}

// One load into LDS: 16 bytes a lane, the wave's 1 KB from `lds` on.
__device__ __forceinline__ void load_lds(u32x4 d, uint32_t from, uint32_t lds) {
  // m0 is the compiler's own, which it warns of: it has to know that its value is gone
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds),
               "v"(from), "s"(d)
               : "memory", "m0");
#pragma clang diagnostic pop
}
__device__ __forceinline__ u32x4 descriptor(const uint8_t* p, int64_t bytes) {
  const uint64_t q = (uint64_t)p;
  // the same in every lane, which the compiler does not always see
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)q),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)(q >> 32)),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)(bytes > 0 ? (uint32_t)bytes : 0u)),
               (uint32_t)kRsrcWord3};
}

// R rows of an operand: their way from memory to LDS, 128 bytes of codes a step of 256 k, by
// `THREADS` threads, and 16 bytes of scales a span of two steps.
template <int R, int THREADS>
struct Side {
  static constexpr int kLoads = R * 128 / (THREADS * 16);  // of a thread, for a step
  static_assert(R * 128 % (THREADS * 16) == 0, "whole loads");
  const uint8_t* codes;  // the tile's first row
  const uint8_t* scales;
  int64_t ld, span;      // bytes of a row, and of a span's scales
  int32_t rows, groups;
  uint32_t off[kLoads];
  int32_t chunk;

  // `count` groups from span `first` on, of rows of `g`.
  __device__ __forceinline__ Side(const uint8_t* c, const uint8_t* s, int64_t row0, int64_t n,
                                  int32_t g, int32_t first, int32_t count, int tid) {
    ld = (int64_t)g * 16;
    span = n * 16;
    codes = c + row0 * ld + (int64_t)first * 256;
    scales = s + row0 * 16 + first * span;
    rows = (int32_t)(n - row0 < R ? n - row0 : R);
    groups = count;
    const int row = tid >> 3;
    chunk = (tid & 7) ^ (row & 7);  // whole eights of rows on, the same
#pragma unroll
    for (int i = 0; i < kLoads; i++) off[i] = (uint32_t)((row + i * (THREADS / 8)) * ld + chunk * 16);
  }
  // The codes of a step, into LDS at `lds` (the wave's part of the first load).  Groups past the
  // end would be the next row's: there a lane reads out of bounds.
  __device__ __forceinline__ void load(int step, uint32_t lds) {
    const int32_t left = groups - step * 8;
    if (left < 8) {
#pragma unroll
      for (int i = 0; i < kLoads; i++) off[i] = chunk < left ? off[i] : 0xfffffff0u;
    }
    const u32x4 d = descriptor(codes + (int64_t)step * 128, left > 0 ? (rows - 1) * ld + left * 16 : 0);
#pragma unroll
    for (int i = 0; i < kLoads; i++) load_lds(d, off[i], lds + i * (THREADS * 16));
  }
};

// What lane `lane` has of fragment f of a half step's rows.
__device__ __forceinline__ i32x4 fragment(const uint8_t* tile, int half, int row0, int f, int lane) {
  const int row = row0 + (lane & 15), chunk = (half * 4 + (lane >> 4)) ^ (row & 7);
  return *(const i32x4*)(tile + row * 128 + chunk * 16 + f * 2048);
}

// Small products: BM x BN tiles, two waves by two, two or three workgroups a compute unit; PARTS > 1:
// k is divided among so many fours of waves, whose sums are added at the end.
template <int DT, int BM, int BN, int PARTS>
__global__ __launch_bounds__(256 * PARTS, 2) void product_kernel(Mx4Args g) {
  constexpr int kThreads = 256;
  constexpr int FM = BM / 32, FN = BN / 32;  // fragments of a wave
  using SideA = Side<BM, kThreads>;
  using SideB = Side<BN, kThreads>;
  constexpr int kTile = (BM + BN) * 128;
  constexpr int kScaleLoads = (BM + BN + kThreads - 1) / kThreads;
  constexpr int kPart = 2 * kTile + kScaleLoads * kThreads * 16;  // bytes of LDS
  static_assert(BM % 64 == 0, "a wave's scales are of one operand");
  static_assert(PARTS == 1 || kPart >= FM * FN * 256 * 16, "a part's sums fit its LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t all_lds[PARTS * kPart];
  const int tid = threadIdx.x & 255, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int part = PARTS > 1 ? __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 8)) : 0;
  uint8_t* const lds = all_lds + part * kPart;
  int32_t tm, tn;
  tile_of(g, &tm, &tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  // every part has as many steps, whose groups need not exist
  const int each = ((g.groups + 15) / 16 + PARTS - 1) / PARTS;
  const int before = part * each * 16 < g.groups ? part * each * 16 : g.groups;
  const int mine = g.groups - before < each * 16 ? g.groups - before : each * 16;
  const int steps = PARTS > 1 ? each * 2 : (g.groups + 7) / 8;
  SideA a(g.a, g.as, m0, g.m, g.groups, before / 16, mine, tid);
  SideB b(g.b, g.bs, n0, g.n, g.groups, before / 16, mine, tid);
  const uint32_t lds_at = (uint32_t)(uintptr_t)(ZS_LDS uint8_t*)lds + wave * 1024;
  const uint8_t* const scale_tile = lds + 2 * kTile;

  // The scales of span p: a load of a thread is 16 bytes, those of one row, A's rows and then B's.
  auto load_scales = [&](int p) {
    const bool there = p * 16 < mine;
    const u32x4 da = descriptor(a.scales + p * a.span, there ? a.rows * 16 : 0);
    const u32x4 db = descriptor(b.scales + p * b.span, there ? b.rows * 16 : 0);
#pragma unroll
    for (int i = 0; i < kScaleLoads; i++) {
      const int row = i * kThreads + wave * 64;
      const uint32_t to = lds_at + 2 * kTile + i * kThreads * 16;
      if (row < BM)
        load_lds(da, (uint32_t)((row + lane) * 16), to);
      else
        load_lds(db, (uint32_t)((row - BM + lane) * 16), to);
    }
  };
  auto load = [&](int step, int stage) {
    a.load(step, lds_at + stage * kTile);
    b.load(step, lds_at + stage * kTile + BM * 128);
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int j = 0; j < FN; j++) acc[i][j] = f32x4{};
  const int ra = (wave >> 1) * (BM / 2), rb = (wave & 1) * (BN / 2);
  uint32_t sa[FM], sb[FN];

  load_scales(0);
  load(0, 0);
  int stage = 0;
  // Step `step`, the first or second of its span.  Its codes have landed for every wave, and
  // every wave has read the step before, whose place takes the loads of the next one.
  auto one = [&](auto SECOND, int step) {
    constexpr int j = decltype(SECOND)::value * 2;
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const uint8_t* tile = lds + stage * kTile;
    if (j == 0) {
#pragma unroll
      for (int i = 0; i < FM; i++)
        sa[i] = *(const uint32_t*)(scale_tile + (ra + i * 16 + (lane & 15)) * 16 + (lane >> 4) * 4);
#pragma unroll
      for (int i = 0; i < FN; i++)
        sb[i] = *(const uint32_t*)(scale_tile + (BM + rb + i * 16 + (lane & 15)) * 16 + (lane >> 4) * 4);
    }
    // every wave has the span's scales: the next one's come
    if (j == 2) load_scales((step >> 1) + 1);
    load(step + 1, stage ^ 1);
    auto half = [&](auto H) {
      constexpr int h = decltype(H)::value;
      i32x4 fb[FN];
#pragma unroll
      for (int k = 0; k < FN; k++) fb[k] = fragment(tile + BM * 128, h, rb, k, lane);
#pragma unroll
      for (int i = 0; i < FM; i++) {
        const i32x4 fa = fragment(tile, h, ra, i, lane);
#pragma unroll
        for (int k = 0; k < FN; k++) acc[i][k] = mfma4<j + h>(fa, fb[k], acc[i][k], sa[i], sb[k]);
      }
    };
    half(std::integral_constant<int, 0>());
    half(std::integral_constant<int, 1>());
    stage ^= 1;
  };
  for (int step = 0; step < steps; step += 2) {
    one(std::integral_constant<int, 0>(), step);
    if (step + 1 < steps) one(std::integral_constant<int, 1>(), step + 1);
  }
  // no load is on its way into LDS any more
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  if constexpr (PARTS > 1) {  // the first part adds the others' sums, in order
    __syncthreads();
    if (part) {
#pragma unroll
      for (int i = 0; i < FM; i++)
#pragma unroll
        for (int k = 0; k < FN; k++) ((f32x4*)lds)[(i * FN + k) * 256 + tid] = acc[i][k];
    }
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int q = 1; q < PARTS; q++)
#pragma unroll
      for (int i = 0; i < FM; i++)
#pragma unroll
        for (int k = 0; k < FN; k++)
          acc[i][k] += ((const f32x4*)(all_lds + q * kPart))[(i * FN + k) * 256 + tid];
  }

  // acc[i][k][r]: feature m0 + ra + i*16 + (lane>>4)*4 + r, token n0 + rb + k*16 + (lane&15)
  const int64_t f0 = m0 + ra + (lane >> 4) * 4, t0 = n0 + rb + (lane & 15);
#pragma unroll
  for (int k = 0; k < FN; k++) {
    elem_t<DT>* out = (elem_t<DT>*)g.c + (t0 + k * 16) * g.ldc + f0;
    const bool there = t0 + k * 16 < g.n;
    if constexpr (DT != ZS_F32) {
      if (m0 + BM <= g.m) {
        // Two fragments' sums change places between the lanes' rows of 16, so that a lane has
        // eight neighbouring features: rows 0 and 2 the first fragment's, 1 and 3 the second's.
        typedef elem_t<DT> v4 __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int i = 0; i < FM; i += 2) {
          const u32x2 x = __builtin_bit_cast(u32x2, __builtin_convertvector(acc[i][k], v4));
          const u32x2 y = __builtin_bit_cast(u32x2, __builtin_convertvector(acc[i + 1][k], v4));
          const auto lo = __builtin_amdgcn_permlane16_swap(x[0], y[0], false, false);
          const auto hi = __builtin_amdgcn_permlane16_swap(x[1], y[1], false, false);
          if (there)
            *(u32x4_any*)(out + i * 16 + (lane >> 4 & 1) * 12) = u32x4{lo[0], hi[0], lo[1], hi[1]};
        }
        continue;
      }
    }
#pragma unroll
    for (int i = 0; i < FM; i++)
      if (there && f0 + i * 16 < g.m) store4<DT>(out + i * 16, g.m - f0 - i * 16, acc[i][k]);
  }
}

// c += a b, c in the accumulation registers, where the compiler would not leave all 256 sums of a
// lane.  It does not know how long the result takes, so settle() has to come before anything
// else touches the sums.
template <int J>
__device__ __forceinline__ void mfma_held(f32x4& c, i32x4 a, i32x4 b, uint32_t sa, uint32_t sb) {
#define ZS_MFMA(bytes)                                                                       \
  asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " bytes " cbsz:4 blgp:4" \
               : "+a"(c)                                                                     \
               : "v"(a), "v"(b), "v"(sa), "v"(sb))
  if constexpr (J == 0)
    ZS_MFMA("op_sel:[0,0,0] op_sel_hi:[0,0,0]");
  else if constexpr (J == 1)
    ZS_MFMA("op_sel:[1,1,0] op_sel_hi:[0,0,0]");
  else if constexpr (J == 2)
    ZS_MFMA("op_sel:[0,0,0] op_sel_hi:[1,1,0]");
  else
    ZS_MFMA("op_sel:[1,1,0] op_sel_hi:[1,1,0]");
#undef ZS_MFMA
}
// The last matrix instruction's result is written (19 wait states after its issue at most).
__device__ __forceinline__ void settle() { asm volatile("s_nop 15\n\ts_nop 3" ::: "memory"); }

// Large products: 256 x 256 tiles, four waves of 128 x 128, one workgroup a compute unit that
// goes on from tile to tile.
template <int DT>
__global__ __launch_bounds__(256, 1) void held_kernel(Mx4Args g) {
  constexpr int B = kBig, F = 8;
  using Part = Side<B, 256>;
  constexpr int kTile = 2 * B * 128, kLoads = 2 * Part::kLoads;
  constexpr int kStashRow = 256 + 16;  // the rows of a column lie on different banks
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kTile + 2 * B * 16 + 4 * 16 * kStashRow];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int spans = (g.groups + 15) / 16;
  const uint32_t lds_at = (uint32_t)(uintptr_t)(ZS_LDS uint8_t*)lds + wave * 1024;
  const uint8_t* const scale_tile = lds + 2 * kTile;
  const int ra = (wave >> 1) * 128, rb = (wave & 1) * 128;

  // the tiles of this workgroup: its die has a contiguous part of them, which go down bands
  // of 8 tiles of tokens; the die's workgroups take neighbouring ones
  const uint32_t total = (uint32_t)g.tiles_m * (uint32_t)g.tiles_n;
  const uint32_t die = blockIdx.x & 7, per = total >> 3, extra = total & 7;
  const uint32_t end = (die + 1) * per + (die + 1 < extra ? die + 1 : extra);
  const uint32_t step = (gridDim.x + 7 - die) >> 3;
  uint32_t id = die * per + (die < extra ? die : extra) + (blockIdx.x >> 3);

  // where the loads are: the tile's rows, and its place in LDS by thread
  uint32_t off[Part::kLoads];
  const int row = tid >> 3, chunk = (tid & 7) ^ (row & 7);
  const int64_t ld = (int64_t)g.groups * 16;
#pragma unroll
  for (int i = 0; i < Part::kLoads; i++) off[i] = (uint32_t)((row + i * 32) * ld + chunk * 16);
  const uint8_t *pa, *pb, *qa, *qb;  // codes and scales of the tile that is loaded
  int32_t rows_a, rows_b;
  auto aim = [&](uint32_t id, int64_t* m0, int64_t* n0) {
    const uint32_t band = id / ((uint32_t)g.tiles_m * 8);
    const uint32_t in = id - band * (uint32_t)g.tiles_m * 8;
    const uint32_t wide = (uint32_t)g.tiles_n - band * 8 < 8 ? (uint32_t)g.tiles_n - band * 8 : 8;
    *m0 = (int64_t)(in / wide) * B;
    *n0 = (int64_t)(band * 8 + in % wide) * B;
  };
  auto aim_loads = [&](uint32_t id) {
    int64_t m0, n0;
    aim(id, &m0, &n0);
    pa = g.a + m0 * ld;
    pb = g.b + n0 * ld;
    qa = g.as + m0 * 16;
    qb = g.bs + n0 * 16;
    rows_a = (int32_t)(g.m - m0 < B ? g.m - m0 : B);
    rows_b = (int32_t)(g.n - n0 < B ? g.n - n0 : B);
  };
  // a step's descriptors, and whether this thread's chunk of it exists
  struct Aim {
    u32x4 a, b;
    bool there;
  };
  auto aim_step = [&](int s, bool any) {
    const int32_t left = g.groups - s * 8;
    Aim r;
    r.a = descriptor(pa + (int64_t)s * 128, any && left > 0 ? (rows_a - 1) * ld + left * 16 : 0);
    r.b = descriptor(pb + (int64_t)s * 128, any && left > 0 ? (rows_b - 1) * ld + left * 16 : 0);
    r.there = chunk < left;
    return r;
  };
  auto load = [&](const Aim& r, int buffer, int i) {
    const int k = i % Part::kLoads;
    const uint32_t from = r.there ? off[k] : 0xfffffff0u;
    load_lds(i < Part::kLoads ? r.a : r.b, from, lds_at + buffer * kTile + (i < Part::kLoads ? 0 : B * 128) + k * 4096);
  };
  auto load_scales = [&](int p, bool any) {
    const u32x4 da = descriptor(qa + p * g.m * 16, any ? rows_a * 16 : 0);
    const u32x4 db = descriptor(qb + p * g.n * 16, any ? rows_b * 16 : 0);
    load_lds(da, (uint32_t)tid * 16, lds_at + 2 * kTile);
    load_lds(db, (uint32_t)tid * 16, lds_at + 2 * kTile + B * 16);
  };

  f32x4 acc[F][F];
#pragma unroll
  for (int i = 0; i < F; i++)
#pragma unroll
    for (int k = 0; k < F; k++) acc[i][k] = f32x4{};
  i32x4 fa[F], fb[F], ga[F], gb[F];
  uint32_t sa[F], sb[F], ta[F], tb[F];
  auto read_scale = [&](uint32_t* s, int row0, int i) {
    s[i] = *(const uint32_t*)(scale_tile + (row0 + i * 16 + (lane & 15)) * 16 + (lane >> 4) * 4);
  };
  // Multiplies fragments xa, xb (instruction J of the span) while the half `half` of the tile at
  // `tile` is read into ya, yb, NEXT: and the next span's scales, and LOADS: starts the loads of
  // a step into `buffer`.  Reads and loads are dealt out between pairs of matrix instructions,
  // which take longer than issuing them; the last eighth has none, so that the last reads
  // have arrived.
  auto multiply = [&](auto JJ, auto NEXT, auto LOADS, i32x4(&xa)[F], i32x4(&xb)[F],
                      i32x4(&ya)[F], i32x4(&yb)[F], const uint8_t* tile, int half, int buffer,
                      const Aim& r) {
    constexpr int J = decltype(JJ)::value;
    constexpr bool kNext = decltype(NEXT)::value;
    constexpr int kPairs = F * F / 2, kSpan = kPairs * 7 / 8, kReads = 2 * F + (kNext ? 2 * F : 0);
    constexpr int n_loads = decltype(LOADS)::value ? kLoads : 0;
#pragma unroll
    for (int x = 0; x < kPairs; x++) {
#pragma unroll
      for (int e = (x * kReads + kSpan - 1) / kSpan;
           e < ((x + 1) * kReads + kSpan - 1) / kSpan && e < kReads; e++) {
        if (e == 0)
          ya[0] = fragment(tile, half, ra, 0, lane);
        else if (e <= F)
          yb[e - 1] = fragment(tile + B * 128, half, rb, e - 1, lane);
        else if (e < 2 * F)
          ya[e - F] = fragment(tile, half, ra, e - F, lane);
        else if (e < 3 * F)
          read_scale(ta, ra, e - 2 * F);
        else
          read_scale(tb, B + rb, e - 3 * F);
      }
#pragma unroll
      for (int e = (x * n_loads + kSpan - 1) / kSpan;
           e < ((x + 1) * n_loads + kSpan - 1) / kSpan && e < n_loads; e++)
        load(r, buffer, e);
#pragma unroll
      for (int y = 2 * x; y < 2 * x + 2; y++) {
        // to and fro, so that a turn keeps both a row's and a column's operand
        const int i = y / F, j = i & 1 ? F - 1 - y % F : y % F;
        mfma_held<J>(acc[i][j], xa[i], xb[j], sa[i], sb[j]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // Every load has landed, and every wave has read what it reads.  Loads and stores complete in
  // the order in which they were issued: a whole tile's stores, which come after the loads
  // waited for, may go on.
  auto meet = [] { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
  constexpr int kStores = DT == ZS_F32 ? 63 : F * 4;  // 64 in fp32, one more than can be asked for
  auto meet_storing = [] {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kStores) : "memory");
  };
  bool storing = false;

  std::integral_constant<int, 0> c0;
  std::integral_constant<int, 1> c1;
  std::integral_constant<int, 2> c2;
  std::integral_constant<int, 3> c3;
  std::integral_constant<bool, false> no;
  std::integral_constant<bool, true> yes;
  if (id >= end) return;
  aim_loads(id);
  load_scales(0, true);
  {
    const Aim r = aim_step(0, true), q = aim_step(1, true);
#pragma unroll
    for (int i = 0; i < kLoads; i++) load(r, 0, i);
#pragma unroll
    for (int i = 0; i < kLoads; i++) load(q, 1, i);
  }
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kLoads) : "memory");
#pragma unroll
  for (int i = 0; i < F; i++) {
    fa[i] = fragment(lds, 0, ra, i, lane);
    fb[i] = fragment(lds + B * 128, 0, rb, i, lane);
    read_scale(ta, ra, i);
    read_scale(tb, B + rb, i);
  }
  const Aim none = {};
  for (; id < end; id += step) {
    const bool more = id + step < end;
    int64_t m0, n0;
    aim(id, &m0, &n0);
    int p = 0;
    do {
      const bool last = p + 1 == spans;
#pragma unroll
      for (int i = 0; i < F; i++) {
        sa[i] = ta[i];
        sb[i] = tb[i];
      }
      multiply(c0, no, no, fa, fb, ga, gb, lds, 1, 0, none);
      // the span's second step is there; its first one's place and the scales' are free
      if (storing)
        meet_storing();
      else
        meet();
      storing = false;
      if (last && more) aim_loads(id + step);
      const bool any = !last || more;
      load_scales(last ? 0 : p + 1, any);
      Aim r = aim_step(last ? 0 : 2 * p + 2, any);
      multiply(c1, no, yes, ga, gb, fa, fb, lds + kTile, 0, 0, r);
      multiply(c2, no, no, fa, fb, ga, gb, lds + kTile, 1, 0, none);
      meet();
      r = aim_step(last ? 1 : 2 * p + 3, any);
      multiply(c3, yes, yes, ga, gb, fa, fb, lds, 0, 1, r);
      settle();
    } while (++p < spans);
    // acc[i][k][r]: feature m0 + ra + i*16 + (lane>>4)*4 + r, token n0 + rb + k*16 + (lane&15)
    const int64_t f0 = m0 + ra + (lane >> 4) * 4, t0 = n0 + rb + (lane & 15);
    elem_t<DT>* out = (elem_t<DT>*)g.c + t0 * g.ldc + f0;
    auto sums = [&](int i, int k) {
      f32x4 x;
#pragma unroll
      for (int r = 0; r < 4; r++)
        asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(x[r]) : "a"(acc[i][k][r]));
      acc[i][k] = f32x4{};
      return x;
    };
    storing = m0 + B <= g.m && n0 + B <= g.n;
    if (!storing) {
#pragma unroll
      for (int k = 0; k < F; k++) {
#pragma unroll
        for (int i = 0; i < F; i++) {
          const f32x4 x = sums(i, k);
          if (t0 + k * 16 < g.n && f0 + i * 16 < g.m) store4<DT>(out + i * 16, g.m - f0 - i * 16, x);
          __builtin_amdgcn_sched_barrier(0);
        }
        out += 16 * g.ldc;
      }
    } else if constexpr (DT == ZS_F32) {
#pragma unroll
      for (int k = 0; k < F; k++) {
#pragma unroll
        for (int i = 0; i < F; i++) {
          store4<DT>(out + i * 16, 4, sums(i, k));
          __builtin_amdgcn_sched_barrier(0);
        }
        out += 16 * g.ldc;
      }
    } else {
      // 16 tokens' rows go through LDS, so that a store has whole lines: four rows of 256 bytes
      typedef elem_t<DT> v4 __attribute__((ext_vector_type(4)));
      uint8_t* const stash = lds + 2 * kTile + 2 * B * 16 + wave * 16 * kStashRow;
      uint8_t* to = stash + (lane & 15) * kStashRow + (lane >> 4) * 8;
      const uint8_t* from = stash + (lane >> 4) * kStashRow + (lane & 15) * 16;
      out = (elem_t<DT>*)g.c + (n0 + rb + (lane >> 4)) * g.ldc + m0 + ra + (lane & 15) * 8;
      auto write = [&](auto NT) {
#pragma unroll
        for (int k = 0; k < F; k++) {
#pragma unroll
          for (int i = 0; i < F; i++)
            *(u32x2*)(to + i * 32) = __builtin_bit_cast(u32x2, __builtin_convertvector(sums(i, k), v4));
#pragma unroll
          for (int i = 0; i < 4; i++)
            st16<decltype(NT)::value>(out + i * 4 * g.ldc, *(const u32x4*)(from + i * 4 * kStashRow));
          __builtin_amdgcn_sched_barrier(0);
          out += 16 * g.ldc;
        }
      };
      if (g.streaming)
        write(yes);
      else
        write(no);
    }
  }
  // no load is on its way into LDS any more
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Few tokens: FM * 16 features a workgroup, FN * 16 tokens, spans of k dealt out over eight waves.
constexpr int kFewWaves = 8;
template <int DT, int FM, int FN>
__global__ __launch_bounds__(kFewWaves * 64) void few_kernel(Mx4Args g) {
  __shared__ f32x4 parts[kFewWaves][FM][FN][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t m0 = (int64_t)blockIdx.x * FM * 16, n0 = (int64_t)blockIdx.y * FN * 16;
  const int64_t ld = (int64_t)g.groups * 16;
  const int spans = (g.groups + 15) / 16;
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int k = 0; k < FN; k++) acc[i][k] = f32x4{};
  // rows that do not exist are the last one's, and go nowhere
  const uint8_t *pa[FM], *pb[FN], *qa[FM], *qb[FN];
#pragma unroll
  for (int i = 0; i < FM; i++) {
    const int64_t row = m0 + i * 16 + (lane & 15) < g.m ? m0 + i * 16 + (lane & 15) : g.m - 1;
    pa[i] = g.a + row * ld + (lane >> 4) * 16;
    qa[i] = g.as + row * 16 + (lane >> 4) * 4;
  }
#pragma unroll
  for (int k = 0; k < FN; k++) {
    const int64_t row = n0 + k * 16 + (lane & 15) < g.n ? n0 + k * 16 + (lane & 15) : g.n - 1;
    pb[k] = g.b + row * ld + (lane >> 4) * 16;
    qb[k] = g.bs + row * 16 + (lane >> 4) * 4;
  }
  for (int p = wave; p < spans; p += kFewWaves) {
    i32x4 fa[FM][4], fb[FN][4];
    uint32_t sa[FM], sb[FN];
    const int left = g.groups - p * 16;
    // a lane's groups past the end are zeros: what is read there is its last one
    auto read = [&](const uint8_t* codes, i32x4(&f)[4]) {
#pragma unroll
      for (int j = 0; j < 4; j++) {
        if (left >= 16) {
          f[j] = *(const i32x4*)(codes + p * 256 + j * 64);
        } else {
          const int group = j * 4 + (lane >> 4), at = group < left ? j * 64 : -(lane >> 4) * 16;
          f[j] = *(const i32x4*)(codes + p * 256 + at);
          if (group >= left) f[j] = i32x4{};
        }
      }
    };
#pragma unroll
    for (int i = 0; i < FM; i++) {
      sa[i] = *(const uint32_t*)(qa[i] + (int64_t)p * g.m * 16);
      read(pa[i], fa[i]);
    }
#pragma unroll
    for (int k = 0; k < FN; k++) {
      sb[k] = *(const uint32_t*)(qb[k] + (int64_t)p * g.n * 16);
      read(pb[k], fb[k]);
    }
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
      for (int k = 0; k < FN; k++) {
        acc[i][k] = mfma4<0>(fa[i][0], fb[k][0], acc[i][k], sa[i], sb[k]);
        acc[i][k] = mfma4<1>(fa[i][1], fb[k][1], acc[i][k], sa[i], sb[k]);
        acc[i][k] = mfma4<2>(fa[i][2], fb[k][2], acc[i][k], sa[i], sb[k]);
        acc[i][k] = mfma4<3>(fa[i][3], fb[k][3], acc[i][k], sa[i], sb[k]);
      }
  }
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int k = 0; k < FN; k++) parts[wave][i][k][lane] = acc[i][k];
  __syncthreads();
  for (int e = tid; e < FM * FN * 64; e += kFewWaves * 64) {
    const int l = e & 63, k = (e >> 6) % FN, i = (e >> 6) / FN;
    f32x4 s = parts[0][i][k][l];
#pragma unroll
    for (int w = 1; w < kFewWaves; w++) s += parts[w][i][k][l];
    const int64_t t = n0 + k * 16 + (l & 15), f = m0 + i * 16 + (l >> 4) * 4;
    if (t < g.n && f < g.m) store4<DT>((elem_t<DT>*)g.c + t * g.ldc + f, g.m - f, s);
  }
}

// Up to so many tokens the weight is streamed, and up to 64 where tiles would leave most of the card
// idle.  us streamed and in tiles, on weights that are not in the caches (tokens x width x
// features): 32 x 4096 x 22016 17 and 18, 48 x 4096 x 22016 (172 tiles) 26 and 18, 64 x 22016 x
// 4096 (32) 26 and 71.  32 features a workgroup where there are workgroups enough, else 16: 16 x
// 4096 x 22016 14 and 16, 16 x 22016 x 4096 21 and 17.
constexpr int64_t kFewTokens = 32;
constexpr int64_t kFewTiles = 96;
constexpr int64_t kCus = 256;
// From so many tiles of 256 x 256 on, the card is filled by them; below, by tiles of 128 x 128
// while there are as many as compute units; else by 128 x 64.  us with large, middle and small
// tiles (tokens x width x features): 4096 x 4096 x 4096 34, 42 and 49; 2048 x 2048 x 6144 (192
// large tiles) 20, 22 and 24; 2048 x 4096 x 4096 (128) 30, 23 and 28; 512 x 4096 x 11008 30, 20
// and 22; 1024 x 4096 x 4096 (256 middle tiles) 29, 15 and 15; 128 x 4096 x 22016 (172) 30, 18
// and 16.
constexpr int64_t kHeldTiles = 192;
// Fewer tiles than this leave half of the card idle; with a long k, from so many groups on, tiles of
// 64 x 64 whose k is divided among the workgroup's waves are faster: 128 x 22016 x 4096 39 us for 72,
// 100 x 28672 x 500 29 for 64, 128 x 2048 x 2048 6.2 for 7.4.
constexpr int64_t kSplitTiles = 128;
constexpr int64_t kSplitGroups = 64;

int check_product(const char* who, const void* x_codes, const void* x_scales, const void* w_codes,
                  const void* w_scales, const void* out, int64_t out_stride, int64_t tokens,
                  int64_t features, int64_t width, int32_t dtype) {
  if (!good_dtype(dtype)) return fail(who, "unknown element type");
  if (tokens < 0 || tokens > kMaxSide || features < 0 || features > kMaxSide || width < 1 ||
      width > kMaxWidth)
    return fail(who, "a size is out of range");
  if (out_stride < features) return fail(who, "a row stride is below the features");
  if (tokens == 0 || features == 0) return ZS_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales || !out) return fail(who, "NULL buffer");
  if (!al(out, elem_bytes(dtype)) || !al(x_codes, 16) || !al(x_scales, 16) || !al(w_codes, 16) ||
      !al(w_scales, 16))
    return fail(who, "a buffer is not aligned to its elements, or codes or scales not to 16 bytes");
  // large tiles, the only ones that so many can be of
  if (((features + kBig - 1) / kBig) * ((tokens + kBig - 1) / kBig) > 0xffffff)
    return fail(who, "too many tiles for one call");
  return ZS_OK;
}

}  // namespace
}  // namespace ops
}  // namespace zs

using namespace zs::ops;

extern "C" int zs_mx4_pack(const void* x, int64_t x_stride, void* codes, void* scales,
                           void* codes_t, void* scales_t, int64_t rows, int64_t width,
                           int32_t dtype, void* stream) {
  const char* who = "zs_mx4_pack";
  if (!good_dtype(dtype)) return fail(who, "unknown element type");
  if (rows < 0 || rows > kMaxSide || width < 1 || width > kMaxWidth)
    return fail(who, "a size is out of range");
  if (codes_t && rows > kMaxWidth) return fail(who, "too many rows to pack along them");
  if ((codes == nullptr) != (scales == nullptr) || (codes_t == nullptr) != (scales_t == nullptr))
    return fail(who, "codes and scales go together");
  if (x_stride < width) return fail(who, "a row stride is below width");
  if (rows == 0) return ZS_OK;
  if (!x || (!codes && !codes_t)) return fail(who, "NULL buffer");
  if (!al(x, elem_bytes(dtype)) || !al(codes, 16) || !al(scales, 16) || !al(codes_t, 16) || !al(scales_t, 16))
    return fail(who, "a buffer is not aligned to its elements, or codes or scales not to 16 bytes");
  const int64_t spans = spans_of(width), spans_t = spans_of(rows);
  const bool nt = dtype != ZS_F32 && streams(rows * width * elem_bytes(dtype));
  if (!codes_t) {
    const int64_t blocks = (rows + 3) / 4 * spans;
    if (blocks > 0xffffff) return fail(who, "too many elements for one call");
    with_dtype(dtype, [&](auto DT) {
      with_bool(nt, [&](auto NT) {
        pack_rows_kernel<decltype(DT)::value, decltype(NT)::value>
            <<<dim3((uint32_t)blocks), dim3(256), 0, (hipStream_t)stream>>>(
                (const elem_t<decltype(DT)::value>*)x, x_stride, (uint8_t*)codes, (uint8_t*)scales,
                rows, width, groups_of(width), (uint32_t)spans);
      });
    });
    return launched(who);
  }
  // blocks past the end too: they write the scales of groups that fill a span up
  const int64_t across = codes ? spans * 2 : (width + 255) / 256;
  const bool large = spans_t * 2 * across >= kLargeBlocks;
  const int64_t down = spans_t * (large ? 2 : 8);
  // a launch has fewer than 2^32 threads
  if (down * across > 0x7fffff) return fail(who, "too many elements for one call");
  with_dtype(dtype, [&](auto DT) {
    constexpr int kDt = decltype(DT)::value;
    with_bool(codes != nullptr, [&](auto ROWS) {
      auto go = [&](auto WAVES) {
        pack_both_kernel<kDt, decltype(ROWS)::value, decltype(WAVES)::value>
            <<<dim3((uint32_t)(down * across)), dim3(decltype(WAVES)::value * 64), 0, (hipStream_t)stream>>>(
                (const elem_t<kDt>*)x, x_stride, (uint8_t*)codes, (uint8_t*)scales, (uint8_t*)codes_t,
                (uint8_t*)scales_t, rows, width, (uint32_t)down);
      };
      if (large)
        go(std::integral_constant<int, 8>());
      else
        go(std::integral_constant<int, 2>());
    });
  });
  return launched(who);
}

extern "C" int zs_mx4_unpack(const void* codes, const void* scales, void* x, int64_t x_stride,
                             int64_t rows, int64_t width, int32_t dtype, void* stream) {
  const char* who = "zs_mx4_unpack";
  if (!good_dtype(dtype)) return fail(who, "unknown element type");
  if (rows < 0 || rows > kMaxSide || width < 1 || width > kMaxWidth)
    return fail(who, "a size is out of range");
  if (x_stride < width) return fail(who, "a row stride is below width");
  if (rows == 0) return ZS_OK;
  if (!codes || !scales || !x) return fail(who, "NULL buffer");
  if (!al(x, elem_bytes(dtype)) || !al(codes, 16) || !al(scales, 16))
    return fail(who, "a buffer is not aligned to its elements, or codes or scales not to 16 bytes");
  const int64_t spans = spans_of(width), blocks = (rows + 3) / 4 * spans;
  if (blocks > 0xffffff) return fail(who, "too many elements for one call");
  const bool nt = dtype != ZS_F32 && streams(rows * width * elem_bytes(dtype));
  with_dtype(dtype, [&](auto DT) {
    with_bool(nt, [&](auto NT) {
      unpack_kernel<decltype(DT)::value, decltype(NT)::value>
          <<<dim3((uint32_t)blocks), dim3(256), 0, (hipStream_t)stream>>>(
              (const uint8_t*)codes, (const uint8_t*)scales, (elem_t<decltype(DT)::value>*)x,
              x_stride, rows, width, groups_of(width), (uint32_t)spans);
    });
  });
  return launched(who);
}

extern "C" size_t zs_mx4_linear_bytes(int64_t tokens, int64_t width) {
  if (tokens < 0 || tokens > kMaxSide || width < 1 || width > kMaxWidth) return 0;
  return up256((size_t)(tokens * groups_of(width)) * 16) + up256((size_t)(spans_of(width) * tokens) * 16) + 256;
}

extern "C" int zs_mx4_linear(const void* x, int64_t x_stride, const void* w_codes,
                             const void* w_scales, void* out, int64_t out_stride, int64_t tokens,
                             int64_t features, int64_t width, int32_t x_dtype, int32_t dtype,
                             void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "zs_mx4_linear";
  const size_t need = zs_mx4_linear_bytes(tokens, width);
  if (need == 0) return fail(who, "a size is out of range");
  if (!workspace || !al(workspace, 256)) return fail(who, "the workspace is NULL or not 256-byte aligned");
  if (workspace_bytes < need) return fail(who, "the workspace is too small");
  if (features == 0) return ZS_OK;
  uint8_t* codes = (uint8_t*)workspace;
  uint8_t* scales = codes + up256((size_t)(tokens * groups_of(width)) * 16);
  // the product's arguments are looked at before anything is enqueued
  if (int rc = check_product(who, codes, scales, w_codes, w_scales, out, out_stride, tokens, features, width, dtype))
    return rc;
  if (int rc = zs_mx4_pack(x, x_stride, codes, scales, nullptr, nullptr, tokens, width, x_dtype, stream))
    return rc;
  return zs_mx4_product(codes, scales, w_codes, w_scales, out, out_stride, tokens, features, width,
                        dtype, stream);
}

extern "C" int zs_mx4_product(const void* x_codes, const void* x_scales, const void* w_codes,
                              const void* w_scales, void* out, int64_t out_stride, int64_t tokens,
                              int64_t features, int64_t width, int32_t dtype, void* stream) {
  const char* who = "zs_mx4_product";
  if (int rc = check_product(who, x_codes, x_scales, w_codes, w_scales, out, out_stride, tokens, features, width, dtype))
    return rc;
  if (tokens == 0 || features == 0) return ZS_OK;
  Mx4Args g{};
  g.a = (const uint8_t*)w_codes;
  g.b = (const uint8_t*)x_codes;
  g.as = (const uint8_t*)w_scales;
  g.bs = (const uint8_t*)x_scales;
  g.m = features;
  g.n = tokens;
  g.groups = (int32_t)groups_of(width);
  g.c = out;
  g.ldc = out_stride;
  // 8192 x 4096 x 22016 (360 MB) 330 us streamed and 357 not, 16384 x 8192 x 8192 (268 MB) 451 and
  // 477, 16384 x 2048 x 8192 143 and 140; smaller outputs are read again from the cache
  g.streaming = streams(tokens * features * elem_bytes(dtype));
  const hipStream_t st = (hipStream_t)stream;
  auto tiles = [&](int64_t bm, int64_t bn) {
    return (features + bm - 1) / bm * ((tokens + bn - 1) / bn);
  };
  if (tokens <= kFewTokens || (tokens <= 64 && tiles(128, 64) < kFewTiles)) {
    with_dtype(dtype, [&](auto DT) {
      constexpr int kDt = decltype(DT)::value;
      auto go = [&](auto FM, auto FN) {
        constexpr int kM = decltype(FM)::value * 16, kN = decltype(FN)::value * 16;
        few_kernel<kDt, kM / 16, kN / 16>
            <<<dim3((uint32_t)((features + kM - 1) / kM), (uint32_t)((tokens + kN - 1) / kN)),
               dim3(kFewWaves * 64), 0, st>>>(g);
      };
      using std::integral_constant;
      if (tiles(32, kFewTokens) >= kCus) {
        if (tokens <= 16)
          go(integral_constant<int, 2>(), integral_constant<int, 1>());
        else
          go(integral_constant<int, 2>(), integral_constant<int, 2>());
      } else if (tokens <= 16) {
        go(integral_constant<int, 1>(), integral_constant<int, 1>());
      } else {
        go(integral_constant<int, 1>(), integral_constant<int, 2>());
      }
    });
    return launched(who);
  }
  const bool held = tiles(kBig, kBig) >= kHeldTiles;
  const bool middle = !held && tiles(128, 128) >= kCus;
  const bool split = !middle && tiles(128, 64) < kSplitTiles && g.groups >= kSplitGroups;
  auto go = [&](auto kernel, int64_t bm, int64_t bn, int threads, int64_t most) {
    g.tiles_m = (int32_t)((features + bm - 1) / bm);
    g.tiles_n = (int32_t)((tokens + bn - 1) / bn);
    kernel<<<dim3((uint32_t)std::min(tiles(bm, bn), most)), dim3(threads), 0, st>>>(g);
  };
  constexpr int64_t kAll = 1ll << 31;
  with_dtype(dtype, [&](auto DT) {
    constexpr int kDt = decltype(DT)::value;
    if (held)
      go(held_kernel<kDt>, kBig, kBig, 256, kCus);
    else if (middle)
      go(product_kernel<kDt, 128, 128, 1>, 128, 128, 256, kAll);
    else if (split)
      go(product_kernel<kDt, 64, 64, 4>, 64, 64, 1024, kAll);
    else
      go(product_kernel<kDt, 128, 64, 1>, 128, 64, 256, kAll);
  });
  return launched(who);
}
