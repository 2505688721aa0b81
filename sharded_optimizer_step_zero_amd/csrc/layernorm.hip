// layernorm.hip -- layer norm with the residual's addition and an output in 16, 8 or 4 bits, and
// its gradient with the sums for the weight and the bias.
//
// Forward, a row at a time: s = x + r (rounded and stored), m = mean s, v = mean (s - m)^2,
// rstd = 1 / sqrt(v + eps), y = (s - m) rstd w + b.  The row stays in registers from the loads
// to the output, so every array is read or written once, and the variance is that of the
// differences (no cancellation whatever the mean), both sums in fp64.
//
// Backward: with h = (s - m) rstd and g = w dy, dx = rstd (g - mean g - h mean(g h)) + ds, dw =
// sum over rows of dy h, db = sum of dy.  Up to 8192 columns a workgroup takes every n-th row,
// keeps its part of dw and db in registers and has the next row's loads under way; a second
// kernel adds the parts in a fixed order.  Wider rows leave no registers for that: there a
// first kernel takes the rows' two means, and a second goes down strips of 2048 columns.
//
// A code or a scale that one bit decides is taken from fp64: the fp32 output is within e =
// (|(s-m) rstd w| + |b|) 2^-21 of y (eight roundings' worth, six are made), so where y - e and
// y + e have one code, or one scale for the group, that is y's; elsewhere the products are
// taken again in fp64 (4e-5 of the chunks).
#include "rows.h"

namespace zs {
namespace ops {
namespace {

constexpr int64_t kMaxWidth = 65536;
constexpr int64_t kMaxBlocks = 0x7fffff;
// Rows up to this width keep their parts of dw and db in registers.
constexpr int64_t kHeldWidth = 8192;
constexpr int64_t kStrip = 2048;  // columns of a workgroup beyond that

template <int DT, bool NT, int NC, int T, int CODE>
__global__ __launch_bounds__(T) void layer_norm_kernel(
    const elem_t<DT>* x, int64_t x_stride, const elem_t<DT>* residual, int64_t residual_stride,
    const elem_t<DT>* __restrict__ weight, const elem_t<DT>* __restrict__ bias, elem_t<DT>* sum,
    int64_t sum_stride, elem_t<DT>* __restrict__ y, int64_t y_stride,
    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, float* __restrict__ mean,
    float* __restrict__ rstd, int64_t rows, int64_t width, float eps, double inv_width, int lanes,
    int rows_per_block, int group_lanes) {
  __shared__ double slots[2][16];
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
  double total = 0.0;
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
#pragma unroll
    for (int i = 0; i < 8; i++) total += (double)s[k][i];
  }
  const double m = row_sum(total, lanes, slots[0]) * inv_width;
  double sq = 0.0;
#pragma unroll
  for (int k = 0; k < NC; k++) {
    const int64_t left = live ? width - (int64_t)(k * lanes + in_row) * 8 : 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const double d = left >= 8 || i < left ? (double)s[k][i] - m : 0.0;
      sq = __builtin_fma(d, d, sq);
    }
  }
  const double variance = row_sum(sq, lanes, slots[1]) * inv_width;
  const double root = inverse_root(variance + (double)eps);
  const float r = (float)root;
  // the mean in two parts: a difference from it is off by two roundings of itself
  const float m_high = (float)m, m_low = (float)(m - (double)m_high);
  if (live && in_row == 0) {
    mean[row] = m_high;
    rstd[row] = r;
  }
  constexpr int kCode = CODE < 0 ? 0 : CODE;
  const int64_t groups = (width + group_lanes * 8 - 1) / (group_lanes * 8);
  if (CODE == ZS_E2M1 && live && groups + in_row < (groups + 15) / 16 * 16)  // 15 at most: one a lane
    scales[scale4_at(row, groups + in_row, rows)] = 127;
#pragma unroll
  for (int k = 0; k < NC; k++) {
    const int64_t chunk = k * lanes + in_row, c = chunk * 8, left = live ? width - c : 0;
    f32x8 v = {}, e = {};
    if (left > 0) {
      const f32x8 w = load8<DT>(weight + c, left);
      const f32x8 b = bias ? load8<DT>(bias + c, left) : f32x8{};
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float p = ((s[k][i] - m_high) - m_low) * r * w[i];
        v[i] = p + b[i];
        e[i] = (__builtin_fabsf(p) + __builtin_fabsf(b[i])) * 0x1p-21f;
      }
      if (y) store8<DT, NT>(y + row * y_stride + c, left, v);
    }
    if (CODE >= 0) {
      // in fp64, to the odd side where fp32 loses anything
      auto again = [&](double factor) {
        f32x8 q = {};
        if (left > 0) {
          const f32x8 w = load8<DT>(weight + c, left);
          const f32x8 b = bias ? load8<DT>(bias + c, left) : f32x8{};
#pragma unroll
          for (int i = 0; i < 8; i++)
            q[i] = side_of(__builtin_fma((widen_again(s[k][i]) - m) * root, (double)w[i], (double)b[i]) * factor);
        }
        return q;
      };
      f32x8 least, most;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float a = __builtin_fabsf(v[i]);
        least[i] = a - e[i] > 0.0f ? a - e[i] : 0.0f;
        most[i] = a + e[i];
      }
      uint32_t byte = scale_byte<kCode>(group_amax(most, group_lanes));
      if (byte != scale_byte<kCode>(group_amax(least, group_lanes))) {  // all of the group's lanes
        const f32x8 q = again(1.0);
        byte = scale_byte<kCode>(group_amax(q, group_lanes));
      }
      const float inv = scale_inverse(byte == 255u ? 127u : byte);
      f32x8 lo, hi;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        lo[i] = (v[i] - e[i]) * inv;
        hi[i] = (v[i] + e[i]) * inv;
      }
      if constexpr (CODE == ZS_E2M1) {
        uint32_t q = encode4(lo, 1.0f);
        if (q != encode4(hi, 1.0f)) q = encode4(again((double)inv), 1.0f);
        if (byte == 255u) q = 0;
        if (live && c < groups * 32) {  // zeros behind the row's end
          *(uint32_t*)(codes + row * groups * 16 + chunk * 4) = q;
          if (chunk % 4 == 0) scales[scale4_at(row, chunk / 4, rows)] = (uint8_t)byte;
        }
      } else {
        u32x2 q = encode8<kCode>(lo);
        const u32x2 other = encode8<kCode>(hi);
        if (q[0] != other[0] || q[1] != other[1]) q = encode8<kCode>(again((double)inv));
        if (byte == 255u) q = u32x2{0, 0};
        if (left > 0) {
          store_codes<NT>(codes + row * width + c, left, q);
          if (chunk % group_lanes == 0) scales[row * groups + chunk / group_lanes] = (uint8_t)byte;
        }
      }
    }
  }
}

// The chunks of a row that the backward pass reads.
template <int DT, int NC>
struct GradRow {
  Chunk<DT> s[NC], dy[NC], ds[NC];
  float mean, rstd;
};

template <int DT, bool NT, int NC, int T>
__global__ __launch_bounds__(T) void layer_norm_grad_kernel(
    const elem_t<DT>* dy, int64_t dy_stride, const elem_t<DT>* sum, int64_t sum_stride,
    const elem_t<DT>* __restrict__ weight, const float* __restrict__ mean,
    const float* __restrict__ rstd, const elem_t<DT>* ds, int64_t ds_stride, elem_t<DT>* dx,
    int64_t dx_stride, float* __restrict__ parts, int64_t part_stride, int64_t rows, int64_t width,
    int lanes, int rows_per_block) {
  __shared__ float slots[2][2][16];
  const int in_row = threadIdx.x & (lanes - 1);
  const int sub = rows_per_block > 1 ? threadIdx.x / lanes : 0;
  const int64_t step = (int64_t)gridDim.x * rows_per_block;
  const float inv_width = 1.0f / (float)width;
  f32x8 w[NC], dw[NC], db[NC];
#pragma unroll
  for (int k = 0; k < NC; k++) {
    const int64_t c = (int64_t)(k * lanes + in_row) * 8;
    w[k] = load8<DT>(weight + c, width - c);
    dw[k] = f32x8{};
    db[k] = f32x8{};
  }
  auto load = [&](int64_t row) {
    GradRow<DT, NC> r;
    const int64_t from = row < rows ? row : rows - 1;  // a row that exists
    r.mean = mean[from];
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
    f32x2 dot = {};
#pragma unroll
    for (int k = 0; k < NC; k++) {
      const int64_t left = row < rows ? width - (int64_t)(k * lanes + in_row) * 8 : 0;
      h[k] = (take8<DT>(now.s[k], left, width) - now.mean) * now.rstd;
      g[k] = take8<DT>(now.dy[k], left, width);  // zeros behind the row's end
      dw[k] += g[k] * h[k];
      db[k] += g[k];
      g[k] *= w[k];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        dot[0] += g[k][i];
        dot[1] += g[k][i] * h[k][i];
      }
    }
    const float mean_g = row_sum(dot[0], lanes, slots[turn][0]) * inv_width;
    const float mean_gh = row_sum(dot[1], lanes, slots[turn][1]) * inv_width;
#pragma unroll
    for (int k = 0; k < NC; k++) {
      const int64_t c = (int64_t)(k * lanes + in_row) * 8, left = row < rows ? width - c : 0;
      const f32x8 v = (g[k] - mean_g - h[k] * mean_gh) * now.rstd + take8<DT>(now.ds[k], left, width);
      store8<DT, NT>(dx + row * dx_stride + c, left, v);
    }
  }
  // narrow rows: the workgroup's rows' parts are added here, in order
  float* part = parts + blockIdx.x * 2 * part_stride;
  if (rows_per_block > 1) {
    __shared__ float all[2][256 * 8];
    store8<ZS_F32>(all[0] + threadIdx.x * 8, 8, dw[0]);
    store8<ZS_F32>(all[1] + threadIdx.x * 8, 8, db[0]);
    __syncthreads();
    if (sub != 0) return;
    for (int i = 1; i < rows_per_block; i++) {
      dw[0] += load8<ZS_F32>(all[0] + (i * lanes + in_row) * 8, 8);
      db[0] += load8<ZS_F32>(all[1] + (i * lanes + in_row) * 8, 8);
    }
  }
#pragma unroll
  for (int k = 0; k < NC; k++) {
    const int64_t c = (int64_t)(k * lanes + in_row) * 8;
    if (c < width) {
      store8<ZS_F32>(part + c, 8, dw[k]);
      store8<ZS_F32>(part + part_stride + c, 8, db[k]);
    }
  }
}

// Wide rows, first: mean g and mean(g h) of each row.
template <int DT>
__global__ __launch_bounds__(1024) void wide_means_kernel(
    const elem_t<DT>* __restrict__ dy, int64_t dy_stride, const elem_t<DT>* __restrict__ sum,
    int64_t sum_stride, const elem_t<DT>* __restrict__ weight, const float* __restrict__ mean,
    const float* __restrict__ rstd, f32x2* __restrict__ means, int64_t width) {
  __shared__ float slots[2][16];
  const int64_t row = blockIdx.x;
  const float m = mean[row], r = rstd[row];
  f32x2 dot = {};
  for (int64_t c = threadIdx.x * 8; c < width; c += 1024 * 8) {
    const int64_t left = width - c;
    const Chunk<DT> a = load_row<DT>(sum + row * sum_stride, c, width);
    const Chunk<DT> b = load_row<DT>(dy + row * dy_stride, c, width);
    const f32x8 h = (take8<DT>(a, left, width) - m) * r;
    const f32x8 g = take8<DT>(b, left, width) * load8<DT>(weight + c, left);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      dot[0] += g[i];
      dot[1] += g[i] * h[i];
    }
  }
  const float inv_width = 1.0f / (float)width;
  const float mean_g = row_sum(dot[0], 1024, slots[0]) * inv_width;
  const float mean_gh = row_sum(dot[1], 1024, slots[1]) * inv_width;
  if (threadIdx.x == 0) means[row] = f32x2{mean_g, mean_gh};
}

// Wide rows, then: a strip of columns down every gridDim.y-th row.
template <int DT, bool NT>
__global__ __launch_bounds__(256) void wide_strip_kernel(
    const elem_t<DT>* dy, int64_t dy_stride, const elem_t<DT>* sum, int64_t sum_stride,
    const elem_t<DT>* __restrict__ weight, const float* __restrict__ mean,
    const float* __restrict__ rstd, const f32x2* __restrict__ means, const elem_t<DT>* ds,
    int64_t ds_stride, elem_t<DT>* dx, int64_t dx_stride, float* __restrict__ parts,
    int64_t part_stride, int64_t rows, int64_t width) {
  const int64_t c = blockIdx.x * kStrip + threadIdx.x * 8, left = width - c;
  if (left <= 0) return;
  const f32x8 w = load8<DT>(weight + c, left);
  f32x8 dw = {}, db = {};
#pragma unroll 2
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const Chunk<DT> a = load_row<DT, NT>(sum + row * sum_stride, c, width);
    const Chunk<DT> b = load_row<DT, NT>(dy + row * dy_stride, c, width);
    Chunk<DT> add = {};
    if (ds) add = load_row<DT, NT>(ds + row * ds_stride, c, width);
    const float m = mean[row], r = rstd[row];
    const f32x2 both = means[row];
    const f32x8 h = (take8<DT>(a, left, width) - m) * r;
    f32x8 g = take8<DT>(b, left, width);
    dw += g * h;
    db += g;
    g *= w;
    store8<DT, NT>(dx + row * dx_stride + c, left, (g - both[0] - h * both[1]) * r + take8<DT>(add, left, width));
  }
  float* part = parts + blockIdx.y * 2 * part_stride;
  store8<ZS_F32>(part + c, 8, dw);
  store8<ZS_F32>(part + part_stride + c, 8, db);
}

// Workgroups of the backward pass, each with a part of dw and db: 1 M floats of parts of each,
// 512 at least and 2048 at most, so that narrow rows leave enough on their way.
int64_t grad_blocks(int64_t rows, int64_t width, const Shape& s) {
  if (width > kHeldWidth) {  // slices of the rows, for each strip
    const int64_t strips = (width + kStrip - 1) / kStrip, slices = 2048 / strips;
    return rows < slices ? rows : slices;
  }
  const int64_t g = (2ll << 20) / width, most = g < 512 ? 512 : g > 2048 ? 2048 : g;
  const int per = s.threads / s.lanes;
  const int64_t need = (rows + per - 1) / per;
  return need < most ? need : most;
}

}  // namespace
}  // namespace ops
}  // namespace zs

using namespace zs::ops;

extern "C" int zs_layer_norm_forward(const void* x, int64_t x_stride, const void* residual,
                                     int64_t residual_stride, const void* weight, const void* bias,
                                     void* sum, int64_t sum_stride, void* y, int64_t y_stride,
                                     void* codes, void* scales, float* mean, float* rstd,
                                     int64_t rows, int64_t width, float eps, int32_t dtype,
                                     int32_t code, int32_t group, void* stream) {
  const char* who = "zs_layer_norm_forward";
  if (!good_dtype(dtype)) return fail(who, "unknown element type");
  if (rows < 0 || rows > 0x7fffffff || width < 1 || width > kMaxWidth)
    return fail(who, "a size is out of range");
  if (!(eps >= 0.0f) || !__builtin_isfinite(eps)) return fail(who, "eps must be finite and not negative");
  if ((codes == nullptr) != (scales == nullptr)) return fail(who, "codes and scales go together");
  if ((residual == nullptr) != (sum == nullptr)) return fail(who, "residual and sum go together");
  if (codes && code == ZS_E2M1) {
    if (group != 32) return fail(who, "the 4-bit form has groups of 32");
  } else if (codes && ((code != ZS_E4M3 && code != ZS_E5M2) || !good_group(group))) {
    return fail(who, "the 8-bit form is e4m3 or e5m2 in groups of 32, 64 or 128");
  }
  if (x_stride < width || (residual && (residual_stride < width || sum_stride < width)) ||
      (y && y_stride < width))
    return fail(who, "a row stride is below width");
  if (rows == 0) return ZS_OK;
  if (!x || !weight || !mean || !rstd) return fail(who, "NULL buffer");
  const int eb = elem_bytes(dtype);
  if (!al(x, eb) || !al(residual, eb) || !al(weight, eb) || !al(bias, eb) || !al(sum, eb) ||
      !al(y, eb) || !al(mean, 4) || !al(rstd, 4) || (code == ZS_E2M1 && !al(codes, 4)))
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
          layer_norm_kernel<decltype(DT)::value, decltype(NT)::value, decltype(NC)::value,
                            decltype(T)::value, decltype(CODE)::value>
              <<<dim3((uint32_t)blocks), dim3(s.threads), 0, (hipStream_t)stream>>>(
                  (const E*)x, x_stride, (const E*)residual, residual_stride, (const E*)weight,
                  (const E*)bias, (E*)sum, sum_stride, (E*)y, y_stride, (uint8_t*)codes,
                  (uint8_t*)scales, mean, rstd, rows, width, eps, 1.0 / (double)width, s.lanes,
                  per, group_lanes);
        };
        if (!codes)
          go(std::integral_constant<int, -1>());
        else if (code == ZS_E2M1)
          go(std::integral_constant<int, ZS_E2M1>());
        else
          with_code(code, go);
      });
    });
  });
  return launched(who);
}

extern "C" size_t zs_layer_norm_backward_bytes(int64_t rows, int64_t width) {
  if (rows < 0 || rows > 0x7fffffff || width < 1 || width > kMaxWidth) return 0;
  const size_t parts = (size_t)grad_blocks(rows, width, shape(width));
  const size_t means = width > kHeldWidth ? up256((size_t)rows * 8) : 0;
  return up256(parts * 2 * part_stride_of(width) * 4) + means + 256;
}

extern "C" int zs_layer_norm_backward(const void* dy, int64_t dy_stride, const void* sum,
                                      int64_t sum_stride, const void* weight, const float* mean,
                                      const float* rstd, const void* grad_sum,
                                      int64_t grad_sum_stride, void* grad_x,
                                      int64_t grad_x_stride, void* grad_weight, void* grad_bias,
                                      int64_t rows, int64_t width, int32_t dtype,
                                      int32_t weight_dtype, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  const char* who = "zs_layer_norm_backward";
  if (!good_dtype(dtype)) return fail(who, "unknown element type");
  if (weight_dtype != dtype && weight_dtype != ZS_F32)
    return fail(who, "the weight's gradient has the weight's type or fp32");
  if (rows < 0 || rows > 0x7fffffff || width < 1 || width > kMaxWidth)
    return fail(who, "a size is out of range");
  if (width > kHeldWidth && rows >= (1ll << 22)) return fail(who, "too many rows for one call");
  if (dy_stride < width || sum_stride < width || grad_x_stride < width ||
      (grad_sum && grad_sum_stride < width))
    return fail(who, "a row stride is below width");
  if (!weight || !grad_weight || (rows && (!dy || !sum || !mean || !rstd || !grad_x)))
    return fail(who, "NULL buffer");
  const int eb = elem_bytes(dtype);
  if (!al(dy, eb) || !al(sum, eb) || !al(weight, eb) || !al(mean, 4) || !al(rstd, 4) ||
      !al(grad_sum, eb) || !al(grad_x, eb) || !al(grad_weight, elem_bytes(weight_dtype)) ||
      !al(grad_bias, elem_bytes(weight_dtype)))
    return fail(who, "a buffer is not aligned to its elements");
  if (!workspace || !al(workspace, 256)) return fail(who, "the workspace is NULL or not 256-byte aligned");
  if (workspace_bytes < zs_layer_norm_backward_bytes(rows, width))
    return fail(who, "the workspace is too small");
  const Shape s = shape(width);
  const int per = s.threads / s.lanes;
  const int64_t blocks = grad_blocks(rows, width, s);
  const int64_t stride = part_stride_of(width);
  const bool nt = dtype != ZS_F32 && streams(rows * width * eb * (grad_sum ? 4 : 3));
  float* parts = (float*)workspace;
  f32x2* means = (f32x2*)((uint8_t*)workspace + up256((size_t)blocks * 2 * stride * 4));
  if (blocks)
    with_dtype(dtype, [&](auto DT) {
      constexpr int kDt = decltype(DT)::value;
      using E = elem_t<kDt>;
      if (width > kHeldWidth)
        wide_means_kernel<kDt><<<dim3((uint32_t)rows), dim3(1024), 0, (hipStream_t)stream>>>(
            (const E*)dy, dy_stride, (const E*)sum, sum_stride, (const E*)weight, mean, rstd, means,
            width);
      with_bool(nt, [&](auto NT) {
        constexpr bool kNt = decltype(NT)::value;
        if (width > kHeldWidth) {
          wide_strip_kernel<kDt, kNt>
              <<<dim3((uint32_t)((width + kStrip - 1) / kStrip), (uint32_t)blocks), dim3(256), 0,
                 (hipStream_t)stream>>>((const E*)dy, dy_stride, (const E*)sum, sum_stride,
                                        (const E*)weight, mean, rstd, means, (const E*)grad_sum,
                                        grad_sum_stride, (E*)grad_x, grad_x_stride, parts, stride,
                                        rows, width);
          return;
        }
        auto go = [&](auto NC, auto T) {
          layer_norm_grad_kernel<kDt, kNt, decltype(NC)::value, decltype(T)::value>
              <<<dim3((uint32_t)blocks), dim3(s.threads), 0, (hipStream_t)stream>>>(
                  (const E*)dy, dy_stride, (const E*)sum, sum_stride, (const E*)weight, mean, rstd,
                  (const E*)grad_sum, grad_sum_stride, (E*)grad_x, grad_x_stride, parts, stride,
                  rows, width, s.lanes, per);
        };
        if (s.threads == 512)
          go(std::integral_constant<int, 2>(), std::integral_constant<int, 512>());
        else if (s.nc == 2)
          go(std::integral_constant<int, 2>(), std::integral_constant<int, 256>());
        else
          go(std::integral_constant<int, 1>(), std::integral_constant<int, 256>());
      });
    });
  if (int rc = launched(who)) return rc;
  with_dtype(weight_dtype, [&](auto WT) {
    using W = elem_t<decltype(WT)::value>;
    columns_kernel<decltype(WT)::value>
        <<<dim3((uint32_t)((width + 31) / 32), grad_bias ? 2 : 1), dim3(1024), 0,
           (hipStream_t)stream>>>(parts, 2 * stride, blocks, (W*)grad_weight, width, stride,
                                  (W*)grad_bias);
  });
  return launched(who);
}
