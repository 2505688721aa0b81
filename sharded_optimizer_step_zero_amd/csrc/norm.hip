// norm.hip -- root-mean-square norm with the residual's addition and an 8-bit
// output, and its gradient.
//
// Forward, a row at a time: s = x + r (rounded and stored), rstd = 1 /
// sqrt(mean(s^2) + eps), y = s * rstd * w.  The row stays in registers between
// the sum of squares and the output, so every array is read or written once; 8
// elements a lane, a row over a workgroup (or a part of one for narrow rows).
// A group's largest magnitude is a maximum over 4, 8 or 16 neighbouring lanes, so
// the 8-bit output needs neither LDS nor a second pass.
//
// Backward: with h = s * rstd, dx = rstd * (w dy - h * mean(w dy h)) + ds.  dw =
// sum over rows of dy h: a workgroup takes every n-th row and keeps its part of dw
// in registers; a second kernel adds the parts in a fixed order.
// The next row's loads are under way while one is worked on.
//
// Both are bound by HBM.  Where a group's largest lies next to the border at which the
// scale steps, the last bit decides a factor of two; so the forward sums its
// squares and takes the root in fp64, which also holds the squares of every finite
// element, rounds rstd once, and takes such groups, and elements next to a tie of their
// code, from products in fp64.  (All products in two parts of fp32 took 172 us for
// 161.)  The backward sums in fp32.  Measured, bf16: forward at 16384 x 8192 with residual and
// codes 160 us for 939 MB (5.9 TB/s), backward at 8192 x 4096 46 + 5 us for 268 MB (5.4
// TB/s; 97 us without the prefetch).
#include "ops.h"

namespace zs {
namespace ops {
namespace {

constexpr int64_t kMaxWidth = 65536;
constexpr int64_t kMaxBlocks = 0x7fffff;
// Workgroups of the backward pass, each with a part of dw: 2 M floats of parts, 512
// at least and 2048 at most, so that narrow rows leave enough on their way.
int64_t backward_groups(int64_t width) {
  const int64_t g = (2ll << 20) / width;
  return g < 512 ? 512 : g > 2048 ? 2048 : g;
}

// How a row is spread: `lanes` threads with nc chunks of 8 each; rows up to 512
// wide share a workgroup of 256.  Two chunks a thread before more threads: at
// 16384 rows of 8192, the forward with 512 threads and 2 chunks takes 165 us, with 256 and 4
// 173 and with 1024 and 1 200.  The backward has the same shape, which serves it up to 8192
// columns (8192 rows: 96 us, 5.6 TB/s); a workgroup of 1024 leaves it 128 registers a lane
// where it needs more, and above it spills inside its loop: 8192 x 12288 732 us, 1.1 TB/s.
struct Shape {
  int lanes, nc, threads;
};
Shape shape(int64_t width) {
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

template <int DT, bool NT, int NC, int T, int CODE>
__global__ __launch_bounds__(T) void norm_kernel(
    const elem_t<DT>* x, int64_t x_stride, const elem_t<DT>* residual, int64_t residual_stride,
    const elem_t<DT>* __restrict__ weight, elem_t<DT>* sum, int64_t sum_stride,
    elem_t<DT>* __restrict__ y, int64_t y_stride, uint8_t* __restrict__ codes,
    uint8_t* __restrict__ scales, float* __restrict__ rstd, int64_t rows, int64_t width,
    float eps, double inv_width, int lanes, int rows_per_block, int group_lanes) {
  __shared__ double slots[16];
  const int in_row = threadIdx.x & (lanes - 1);
  const int64_t row = (int64_t)blockIdx.x * rows_per_block + (rows_per_block > 1 ? threadIdx.x / lanes : 0);
  const bool live = row < rows;  // no early return: the shuffles and barriers are the workgroup's
  const int64_t from = live ? row : rows - 1;  // a row that exists
  Chunk<DT> in[NC], add[NC];
#pragma unroll
  for (int k = 0; k < NC; k++) {
    const int64_t c = (int64_t)(k * lanes + in_row) * 8;
    in[k] = load_row<DT, NT>(x + from * x_stride, c, width);
    if (residual) add[k] = load_row<DT, NT>(residual + from * residual_stride, c, width);
  }
  f32x8 s[NC];
  double sq = 0.0;
#pragma unroll
  for (int k = 0; k < NC; k++) {
    const int64_t c = (int64_t)(k * lanes + in_row) * 8, left = live ? width - c : 0;
    s[k] = take8<DT>(in[k], left, width);
    if (residual) {
      s[k] += take8<DT>(add[k], left, width);
      // the stored, rounded sum is what is normalised
      s[k] = __builtin_convertvector(__builtin_convertvector(s[k], typename Elem<DT>::vec), f32x8);
      store8<DT, NT>(sum + row * sum_stride + c, left, s[k]);
    }
    // a square of 24 bits is exact in fp64, and finite whatever the element
#pragma unroll
    for (int i = 0; i < 8; i++) sq = __builtin_fma((double)s[k][i], (double)s[k][i], sq);
  }
  const double total = row_sum(sq, lanes, slots);
  const double root = inverse_root(__builtin_fma(total, inv_width, (double)eps));
  const float r = (float)root;
  if (live && in_row == 0) rstd[row] = r;
  const int64_t groups = (width + group_lanes * 8 - 1) / (group_lanes * 8);
#pragma unroll
  for (int k = 0; k < NC; k++) {
    const int64_t chunk = k * lanes + in_row, c = chunk * 8, left = live ? width - c : 0;
    f32x8 v = {};
    if (left > 0) {
      v = s[k] * r * load8<DT>(weight + c, left);
      if (y) store8<DT, NT>(y + row * y_stride + c, left, v);
    }
    if (CODE >= 0) {
      float amax = group_amax(v, group_lanes);
      if ((__float_as_uint(amax) & 0x7fffffu) - 0x5ffffdu <= 6u) {
        // within three units (three roundings make two and a quarter there) of 1.75 times a
        // power of two, where the scale steps: the group again with its products in fp64
        // (all of its lanes come here)
        if (left > 0) {
          const f32x8 wt = load8<DT>(weight + c, left);
#pragma unroll
          for (int i = 0; i < 8; i++)
            v[i] = side_of(widen_again(s[k][i]) * root * (double)wt[i]);
        }
        amax = group_amax(v, group_lanes);
      }
      constexpr int kCode = CODE < 0 ? 0 : CODE;
      const uint32_t byte = scale_byte<kCode>(amax);
      const float inv = scale_inverse(byte == 255u ? 127u : byte);
      // The products are off by three roundings, and these two by one more: where what lies
      // 2^-21 (four units or more) below and above has one code, that is the element's, normal or subnormal.
      const float below = inv * (1.0f - 0x1p-21f), above = inv * (1.0f + 0x1p-21f);
      f32x8 lo, hi;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        lo[i] = v[i] * below;
        hi[i] = v[i] * above;
      }
      u32x2 w = encode8<kCode>(lo);
      const u32x2 other = encode8<kCode>(hi);
      if ((w[0] != other[0] || w[1] != other[1]) && left > 0) {  // from products in fp64
        const f32x8 wt = load8<DT>(weight + c, left);
#pragma unroll
        for (int i = 0; i < 8; i++)
          lo[i] = side_of(widen_again(s[k][i]) * root * (double)wt[i] * (double)inv);
        w = encode8<kCode>(lo);
      }
      if (byte == 255u) w = u32x2{0, 0};
      if (left > 0) {
        store_codes<NT>(codes + row * width + c, left, w);
        if (chunk % group_lanes == 0) scales[row * groups + chunk / group_lanes] = (uint8_t)byte;
      }
    }
  }
}

// The chunks of a row that the backward pass reads.
template <int DT, int NC>
struct GradRow {
  Chunk<DT> s[NC], dy[NC], ds[NC];
  float rstd;
};

template <int DT, bool NT, int NC, int T>
__global__ __launch_bounds__(T) void norm_grad_kernel(
    const elem_t<DT>* dy, int64_t dy_stride, const elem_t<DT>* sum, int64_t sum_stride,
    const elem_t<DT>* __restrict__ weight, const float* __restrict__ rstd,
    const elem_t<DT>* ds, int64_t ds_stride, elem_t<DT>* dx, int64_t dx_stride,
    float* __restrict__ parts, int64_t part_stride, int64_t rows, int64_t width, int lanes,
    int rows_per_block) {
  __shared__ float slots[2][16];
  const int in_row = threadIdx.x & (lanes - 1);
  const int sub = rows_per_block > 1 ? threadIdx.x / lanes : 0;
  const int64_t step = (int64_t)gridDim.x * rows_per_block;
  const float inv_width = 1.0f / (float)width;
  f32x8 w[NC], dw[NC];
#pragma unroll
  for (int k = 0; k < NC; k++) {
    const int64_t c = (int64_t)(k * lanes + in_row) * 8;
    w[k] = load8<DT>(weight + c, width - c);
    dw[k] = f32x8{};
  }
  auto load = [&](int64_t row) {
    GradRow<DT, NC> r;
    const int64_t from = row < rows ? row : rows - 1;  // a row that exists
    r.rstd = rstd[from];
#pragma unroll
    for (int k = 0; k < NC; k++) {
      const int64_t c = (int64_t)(k * lanes + in_row) * 8;
      r.s[k] = load_row<DT, NT>(sum + from * sum_stride, c, width);
      r.dy[k] = load_row<DT, NT>(dy + from * dy_stride, c, width);
      r.ds[k] = Chunk<DT>{};
      if (ds) r.ds[k] = load_row<DT, NT>(ds + from * ds_stride, c, width);
    }
    return r;
  };
  int turn = 0;
  const int64_t first = (int64_t)blockIdx.x * rows_per_block;
  GradRow<DT, NC> next = load(first + sub);
  for (int64_t row0 = first; row0 < rows; row0 += step, turn ^= 1) {
    const GradRow<DT, NC> now = next;
    const int64_t row = row0 + sub;
    // the next row is on its way while this one is worked on
    if (row0 + step < rows) next = load(row + step);
    f32x8 h[NC], g[NC];
    float dot = 0.0f;
#pragma unroll
    for (int k = 0; k < NC; k++) {
      const int64_t left = row < rows ? width - (int64_t)(k * lanes + in_row) * 8 : 0;
      h[k] = take8<DT>(now.s[k], left, width) * now.rstd;
      g[k] = take8<DT>(now.dy[k], left, width);
      dw[k] += g[k] * h[k];
      g[k] *= w[k];
#pragma unroll
      for (int i = 0; i < 8; i++) dot += g[k][i] * h[k][i];
    }
    const float mean = row_sum(dot, lanes, slots[turn]) * inv_width;
#pragma unroll
    for (int k = 0; k < NC; k++) {
      const int64_t c = (int64_t)(k * lanes + in_row) * 8, left = row < rows ? width - c : 0;
      const f32x8 v = (g[k] - h[k] * mean) * now.rstd + take8<DT>(now.ds[k], left, width);
      store8<DT, NT>(dx + row * dx_stride + c, left, v);
    }
  }
  // narrow rows: the workgroup's rows' parts are added here, in order
  float* part = parts + blockIdx.x * part_stride;
  if (rows_per_block > 1) {
    __shared__ float all[256 * 8];
    store8<ZS_F32>(all + threadIdx.x * 8, 8, dw[0]);
    __syncthreads();
    if (sub != 0) return;
    for (int i = 1; i < rows_per_block; i++)
      dw[0] += load8<ZS_F32>(all + (i * lanes + in_row) * 8, 8);
  }
#pragma unroll
  for (int k = 0; k < NC; k++) {
    const int64_t c = (int64_t)(k * lanes + in_row) * 8;
    if (c < width) store8<ZS_F32>(part + c, 8, dw[k]);
  }
}

// dw[c] = the sum of the parts' column c: 32 slices of the parts a workgroup, each
// in order, then the slices in order.
template <int WT>
__global__ __launch_bounds__(1024) void columns_kernel(const float* __restrict__ parts,
                                                       int64_t part_stride, int64_t n_parts,
                                                       elem_t<WT>* __restrict__ dw,
                                                       int64_t width) {
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

// Workgroups of the backward pass, and parts of dw.
int64_t grad_blocks(int64_t rows, int64_t width, const Shape& s) {
  const int per = s.threads / s.lanes;
  const int64_t need = (rows + per - 1) / per, most = backward_groups(width);
  return need < most ? need : most;
}

int64_t part_stride_of(int64_t width) { return (width + 7) / 8 * 8; }

}  // namespace
}  // namespace ops
}  // namespace zs

using namespace zs::ops;

extern "C" int zs_norm_forward(const void* x, int64_t x_stride, const void* residual,
                               int64_t residual_stride, const void* weight, void* sum,
                               int64_t sum_stride, void* y, int64_t y_stride, void* codes,
                               void* scales, float* rstd, int64_t rows, int64_t width, float eps,
                               int32_t dtype, int32_t code, int32_t group, void* stream) {
  const char* who = "zs_norm_forward";
  if (!good_dtype(dtype)) return fail(who, "unknown element type");
  if (rows < 0 || rows > 0x7fffffff || width < 1 || width > kMaxWidth)
    return fail(who, "a size is out of range");
  if (!(eps >= 0.0f) || !__builtin_isfinite(eps)) return fail(who, "eps must be finite and not negative");
  if ((codes == nullptr) != (scales == nullptr)) return fail(who, "codes and scales go together");
  if ((residual == nullptr) != (sum == nullptr)) return fail(who, "residual and sum go together");
  if (codes && ((code != ZS_E4M3 && code != ZS_E5M2) || !good_group(group)))
    return fail(who, "the 8-bit form is e4m3 or e5m2 in groups of 32, 64 or 128");
  if (x_stride < width || (residual && (residual_stride < width || sum_stride < width)) ||
      (y && y_stride < width))
    return fail(who, "a row stride is below width");
  if (rows == 0) return ZS_OK;
  if (!x || !weight || !rstd) return fail(who, "NULL buffer");
  const int eb = elem_bytes(dtype);
  if (!al(x, eb) || !al(residual, eb) || !al(weight, eb) || !al(sum, eb) || !al(y, eb) ||
      !al(rstd, 4))
    return fail(who, "a buffer is not aligned to its elements");
  const Shape s = shape(width);
  const int per = s.threads / s.lanes;
  const int64_t blocks = (rows + per - 1) / per;
  // a launch has fewer than 2^32 threads
  if (blocks > kMaxBlocks || blocks * s.threads > 0xffffffffll)
    return fail(who, "too many rows for one call");
  const bool nt = dtype != ZS_F32 && streams(rows * width * ((residual ? 3 : 1) * eb + (y ? eb : 0) + (codes ? 1 : 0)));
  const int group_lanes = codes ? group / 8 : 16;
  with_dtype(dtype, [&](auto DT) {
    with_bool(nt, [&](auto NT) {
      with_shape(s, [&](auto NC, auto T) {
        auto go = [&](auto CODE) {
          using E = elem_t<decltype(DT)::value>;
          norm_kernel<decltype(DT)::value, decltype(NT)::value, decltype(NC)::value,
                      decltype(T)::value,
                      decltype(CODE)::value>
              <<<dim3((uint32_t)blocks), dim3(s.threads), 0, (hipStream_t)stream>>>(
                  (const E*)x, x_stride, (const E*)residual, residual_stride, (const E*)weight,
                  (E*)sum, sum_stride, (E*)y, y_stride, (uint8_t*)codes, (uint8_t*)scales, rstd,
                  rows, width, eps, 1.0 / (double)width, s.lanes, per, group_lanes);
        };
        if (!codes)
          go(std::integral_constant<int, -1>());
        else
          with_code(code, go);
      });
    });
  });
  return launched(who);
}

extern "C" size_t zs_norm_backward_bytes(int64_t rows, int64_t width) {
  if (rows < 0 || rows > 0x7fffffff || width < 1 || width > kMaxWidth) return 0;
  const Shape s = shape(width);
  const size_t parts = (size_t)grad_blocks(rows, width, s);
  return up256(parts * part_stride_of(width) * 4) + 256;
}

extern "C" int zs_norm_backward(const void* dy, int64_t dy_stride, const void* sum,
                                int64_t sum_stride, const void* weight, const float* rstd,
                                const void* grad_sum, int64_t grad_sum_stride, void* grad_x,
                                int64_t grad_x_stride, void* grad_weight, int64_t rows,
                                int64_t width, int32_t dtype, int32_t weight_dtype,
                                void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "zs_norm_backward";
  if (!good_dtype(dtype)) return fail(who, "unknown element type");
  if (weight_dtype != dtype && weight_dtype != ZS_F32)
    return fail(who, "the weight's gradient has the weight's type or fp32");
  if (rows < 0 || rows > 0x7fffffff || width < 1 || width > kMaxWidth)
    return fail(who, "a size is out of range");
  if (dy_stride < width || sum_stride < width || grad_x_stride < width ||
      (grad_sum && grad_sum_stride < width))
    return fail(who, "a row stride is below width");
  if (!weight || !grad_weight || (rows && (!dy || !sum || !rstd || !grad_x)))
    return fail(who, "NULL buffer");
  const int eb = elem_bytes(dtype);
  if (!al(dy, eb) || !al(sum, eb) || !al(weight, eb) || !al(rstd, 4) || !al(grad_sum, eb) ||
      !al(grad_x, eb) || !al(grad_weight, elem_bytes(weight_dtype)))
    return fail(who, "a buffer is not aligned to its elements");
  if (!workspace || !al(workspace, 256)) return fail(who, "the workspace is NULL or not 256-byte aligned");
  if (workspace_bytes < zs_norm_backward_bytes(rows, width))
    return fail(who, "the workspace is too small");
  const Shape s = shape(width);
  const int per = s.threads / s.lanes;
  const int64_t blocks = grad_blocks(rows, width, s);
  const int64_t stride = part_stride_of(width);
  const bool nt = dtype != ZS_F32 && streams(rows * width * eb * (grad_sum ? 4 : 3));
  if (blocks)
    with_dtype(dtype, [&](auto DT) {
      with_bool(nt, [&](auto NT) {
        with_shape(s, [&](auto NC, auto T) {
          using E = elem_t<decltype(DT)::value>;
          norm_grad_kernel<decltype(DT)::value, decltype(NT)::value, decltype(NC)::value,
                      decltype(T)::value>
              <<<dim3((uint32_t)blocks), dim3(s.threads), 0, (hipStream_t)stream>>>(
                  (const E*)dy, dy_stride, (const E*)sum, sum_stride, (const E*)weight, rstd,
                  (const E*)grad_sum, grad_sum_stride, (E*)grad_x, grad_x_stride,
                  (float*)workspace, stride, rows, width, s.lanes, per);
        });
      });
    });
  if (int rc = launched(who)) return rc;
  with_dtype(weight_dtype, [&](auto WT) {
    columns_kernel<decltype(WT)::value>
        <<<dim3((uint32_t)((width + 31) / 32)), dim3(1024), 0, (hipStream_t)stream>>>(
            (const float*)workspace, stride, blocks, (elem_t<decltype(WT)::value>*)grad_weight,
            width);
  });
  return launched(who);
}
