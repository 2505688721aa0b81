// rows.h -- what the norms share: a row held in a workgroup's registers, sums over a row,
// roots and sides of borders in fp64, and the columns' sums of a weight's gradient.
#pragma once

#include "ops.h"

namespace zs {
namespace ops {
namespace {

// How a row is spread: `lanes` threads with nc chunks of 8 each; rows up to 512
// wide share a workgroup of 256.  Two chunks a thread before more threads: at
// 16384 rows of 8192, the forward with 512 threads and 2 chunks takes 165 us, with 256 and 4
// 173 and with 1024 and 1 200.  The backward has the same shape, which serves it up to 8192
// columns (8192 rows: 96 us, 5.6 TB/s); a workgroup of 1024 leaves it 128 registers a lane
// where it needs more, and above it spills inside its loop: 8192 x 12288 732 us, 1.1 TB/s.
struct Shape {
  int lanes, nc, threads;
};
inline Shape shape(int64_t width) {
  const int64_t chunks = (width + 7) / 8;
  if (chunks <= 64) {
    int lanes = 16;
    while (lanes < chunks) lanes *= 2;
    return {lanes, 1, 256};
  }
  if (chunks <= 128) return {128, 1, 128};
  int nc = chunks <= 256 ? 1 : 2, lanes = 256;
  while (lanes < 1024 && nc * lanes < chunks) lanes *= 2;
  while (nc * lanes < chunks) nc *= 2;
  return {lanes, nc, lanes};
}

// Sum over the row's threads: within a wave by shuffles, across waves through LDS
// (each call its own slots, written before and read after one barrier).
template <typename F>
__device__ __forceinline__ F row_sum(F x, int lanes, F* slots) {
  const int w = lanes < 64 ? lanes : 64;
  for (int d = 1; d < w; d <<= 1) x += __shfl_xor(x, d, 64);
  if (lanes <= 64) return x;
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = x;
  __syncthreads();
  F s = 0;
  for (int i = 0; i < lanes / 64; i++) s += slots[i];
  return s;
}

// 1 / sqrt(v) in fp64: the hardware's fp32 estimate, of v brought within fp32's range (squares
// reach from 2^-298 to 2^256, and their mean a little below), and two Newton steps; the
// estimate alone where a step has no meaning (0, infinity, NaN).
__device__ __forceinline__ double inverse_root(double v) {
  const bool tiny = v < 0x1p-100, huge = v > 0x1p100;
  v *= tiny ? 0x1p210 : huge ? 0x1p-180 : 1.0;
  double r = __builtin_amdgcn_rsqf((float)v);
  if (!(r > 0.0 && r < __builtin_inf())) return r;
  r *= __builtin_fma(-0.5 * v * r, r, 1.5);
  r *= __builtin_fma(-0.5 * v * r, r, 1.5);
  return r * (tiny ? 0x1p105 : huge ? 0x1p-90 : 1.0);
}

// x in fp64, made anew: a branch that is hardly ever taken must not have the values that the
// squares were made of held for it (34 registers more: 196 us for 158 at 16384 x 8192).
__device__ __forceinline__ double widen_again(float x) {
  asm("" : "+v"(x));
  return (double)x;
}
// d in fp32, cut and its last bit set where that lost anything (rounded to odd): it lies on the
// same side of every value of fewer bits as d, so rounding it again rounds d.
__device__ __forceinline__ float side_of(double d) {
  const float f = (float)d;
  uint32_t u = __float_as_uint(f);
  if ((double)f != d && d == d) u = (u - (__builtin_fabs((double)f) > __builtin_fabs(d) ? 1u : 0u)) | 1u;
  return __uint_as_float(u);
}

// dw[c] = the sum of the parts' column c (a second sum's parts lie `offset` on in each, and
// blockIdx.y 1 adds them into db): 32 slices of the parts a workgroup, each
// in order, then the slices in order.
template <int WT>
__global__ __launch_bounds__(1024) void columns_kernel(const float* __restrict__ parts,
                                                       int64_t part_stride, int64_t n_parts,
                                                       elem_t<WT>* __restrict__ dw,
                                                       int64_t width, int64_t offset = 0,
                                                       elem_t<WT>* __restrict__ db = nullptr) {
  if (blockIdx.y) {
    parts += offset;
    dw = db;
  }
  __shared__ float slots[32][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  const int64_t per = (n_parts + 31) / 32, begin = slice * per;
  const int64_t end = begin + per < n_parts ? begin + per : n_parts;
  float s = 0.0f;
  if (c < width) {
#pragma unroll 8
    for (int64_t p = begin; p < end; p++) s += parts[p * part_stride + c];
  }
  slots[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < width) {
    s = 0.0f;
    for (int i = 0; i < 32; i++) s += slots[i][lane];
    dw[c] = (elem_t<WT>)s;
  }
}

// Calls f with the chunks a thread and the largest workgroup as constants.
template <typename F>
void with_shape(const Shape& s, F f) {
  using std::integral_constant;
  if (s.threads <= 256) {
    if (s.nc == 1)
      f(integral_constant<int, 1>(), integral_constant<int, 256>());
    else
      f(integral_constant<int, 2>(), integral_constant<int, 256>());
  } else if (s.threads == 512) {
    f(integral_constant<int, 2>(), integral_constant<int, 512>());
  } else if (s.nc == 2) {
    f(integral_constant<int, 2>(), integral_constant<int, 1024>());
  } else if (s.nc == 4) {
    f(integral_constant<int, 4>(), integral_constant<int, 1024>());
  } else {
    f(integral_constant<int, 8>(), integral_constant<int, 1024>());
  }
}

inline int64_t part_stride_of(int64_t width) { return (width + 7) / 8 * 8; }

}  // namespace
}  // namespace ops
}  // namespace zs
