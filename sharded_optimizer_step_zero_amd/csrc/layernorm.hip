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
// Codes come from an output in fp64 (whose instructions take no longer than fp32's), rounded to
// fp32 to nearest and, where that may have crossed the border between two codes or two scales, to
// the odd side, so that each code is one rounding of y.  (The output in fp32 with an error bound,
// and both of its ends encoded, took 260 us for 203.)
//
// Bound by HBM.  Measured, bf16, among other calls: forward at 16384 x 8192 with residual and 8-bit
// codes 178 to 192 us for 943 MB, by where its arrays lie (5.3 to 4.9 TB/s; the vector unit is busy for
// three quarters of it), in 4 bits 173; backward at 32768 x 2048 96 us for 537 MB (5.6 TB/s), 16384 x
// 8192 186 us (5.8), 8192 x 12288 in two passes 216 us.  Above 32768 columns a thread has eight chunks
// and spills registers: with residual, in 16 and in 8 bits, 4096 x 32768 185 and 210 us, 4096 x 49152
// 420 and 1350, 4096 x 65536 730 and 690.
#include "rows.h"

namespace zs {
namespace ops {
namespace {

constexpr int64_t kMaxWidth = 65536;
constexpr int64_t kMaxBlocks = 0x7fffff;
// Rows up to this width keep their parts of dw and db in registers.
constexpr int64_t kHeldWidth = 8192;
constexpr int64_t kStrip = 2048;  // columns of a workgroup beyond that

template <int DT>
struct RowArgs {
  const elem_t<DT>*x, *residual, *weight, *bias;
  elem_t<DT>*sum, *y;
  int64_t x_stride, residual_stride, sum_stride, y_stride;
  uint8_t *codes, *scales;
  float *mean, *rstd;
  int64_t rows;
  int32_t width, lanes, rows_per_block, code, group_lanes;
  float eps;
  double inv_width;
};

// Sums and maxima over lanes by moves inside the vector unit (the LDS ways of a shuffle wait some
// hundred cycles each, of which a row has fourteen in a chain: forward at 16384 x 8192 195 us for
// 183, at 32768 x 2048 115 for 98, backward there 101 for 96).

// x of another lane of the row of 16: CTRL 0xb1 lane ^ 1, 0x4e lane ^ 2, 0x141 the other end of the
// eight, 0x140 of the sixteen.
template <int CTRL, typename F>
__device__ __forceinline__ F other_lane(F x) {
  uint32_t w[sizeof(F) / 4];
  __builtin_memcpy(w, &x, sizeof(F));
#pragma unroll
  for (size_t i = 0; i < sizeof(F) / 4; i++)
    w[i] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[i], CTRL, 0xf, 0xf, true);
  __builtin_memcpy(&x, w, sizeof(F));
  return x;
}
// Joins x over n neighbouring lanes, n = 1, 2, 4, 8 or 16.
template <typename F, typename JOIN>
__device__ __forceinline__ F join_lanes(F x, int n, JOIN join) {
  if (n >= 2) x = join(x, other_lane<0xb1>(x));
  if (n >= 4) x = join(x, other_lane<0x4e>(x));
  if (n >= 8) x = join(x, other_lane<0x141>(x));
  if (n >= 16) x = join(x, other_lane<0x140>(x));
  return x;
}
// The sum over 16, 32 or 64 lanes, in all of them.
template <typename F>
__device__ __forceinline__ F wave_sum(F x, int lanes) {
  x = join_lanes(x, 16, [](F a, F b) { return a + b; });
  constexpr int kWords = sizeof(F) / 4;
  uint32_t a[kWords], b[kWords];
  F p, q;
  if (lanes >= 32) {  // rows of 16 change places: 0 and 1, 2 and 3
    __builtin_memcpy(a, &x, sizeof(F));
#pragma unroll
    for (int i = 0; i < kWords; i++) {
      const auto s = __builtin_amdgcn_permlane16_swap(a[i], a[i], false, false);
      a[i] = s[0];
      b[i] = s[1];
    }
    __builtin_memcpy(&p, a, sizeof(F));
    __builtin_memcpy(&q, b, sizeof(F));
    x = p + q;
  }
  if (lanes >= 64) {  // halves of the wave
    __builtin_memcpy(a, &x, sizeof(F));
#pragma unroll
    for (int i = 0; i < kWords; i++) {
      const auto s = __builtin_amdgcn_permlane32_swap(a[i], a[i], false, false);
      a[i] = s[0];
      b[i] = s[1];
    }
    __builtin_memcpy(&p, a, sizeof(F));
    __builtin_memcpy(&q, b, sizeof(F));
    x = p + q;
  }
  return x;
}
// The sum over a row's threads, of which `base` is the first wave: through LDS where they are more
// than a wave (each call its own slots, written before and read after one barrier).
template <typename F>
__device__ __forceinline__ F sum_row(F x, int lanes, int base, F* slots) {
  x = wave_sum(x, lanes);
  if (lanes <= 64) return x;
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = x;
  __syncthreads();
  const int n = lanes / 64;
  return join_lanes(slots[base + (threadIdx.x & (n - 1))], n, [](F a, F b) { return a + b; });
}
// The largest magnitude of a group of 4, 8 or 16 lanes' elements.
__device__ __forceinline__ float amax_lanes(f32x8 x, int lanes) {
  return __uint_as_float(join_lanes(amax_bits(x), lanes, [](uint32_t a, uint32_t b) { return a > b ? a : b; }));
}

// The scale byte of a group, by the format as a value.
__device__ __forceinline__ uint32_t scale_byte_of(int code, float amax) {
  return code == ZS_E4M3 ? scale_byte<ZS_E4M3>(amax)
                         : code == ZS_E5M2 ? scale_byte<ZS_E5M2>(amax) : scale_byte<ZS_E2M1>(amax);
}

// Differences from the mean may pass fp32's range where the elements do not.  Some difference is
// above 2^127 only where the deviation is above 2^119 (65536 columns): such rows' differences are
// taken in quarters, which are exact there, and times four times the deviation's inverse, which
// is then a normal number too.
template <int DT>
__device__ __forceinline__ bool far_apart(float rstd) {
  return DT != ZS_F16 && rstd < 0x1p-110f;
}

// WHOLE: the threads' chunks cover the row exactly.
template <int DT, bool NT, int NC, bool CODES, bool WHOLE>
__device__ __forceinline__ void layer_norm_rows(const RowArgs<DT>& g, double (&slots)[2][16]) {
  const int lanes = g.lanes, width = g.width;
  const int in_row = threadIdx.x & (lanes - 1);
  const int64_t row = (int64_t)blockIdx.x * g.rows_per_block + (g.rows_per_block > 1 ? threadIdx.x / lanes : 0);
  const bool live = row < g.rows;  // no early return: the shuffles and barriers are the workgroup's
  const int64_t from = live ? row : g.rows - 1;  // a row that exists
  // elements of chunk k that exist
  auto count = [&](int k) {
    const int left = width - (k * lanes + in_row) * 8;
    return WHOLE ? 8 : left;
  };
  Chunk<DT> in[NC], add[NC];
#pragma unroll
  for (int k = 0; k < NC; k++) {
    const int c = (k * lanes + in_row) * 8;
    if (WHOLE) {
      in[k] = load_chunk<DT, NT>(g.x + from * g.x_stride + c, 8);
      if (g.residual) add[k] = load_chunk<DT, NT>(g.residual + from * g.residual_stride + c, 8);
    } else {
      in[k] = load_row<DT, NT>(g.x + from * g.x_stride, c, width);
      if (g.residual) add[k] = load_row<DT, NT>(g.residual + from * g.residual_stride, c, width);
    }
  }
  f32x8 s[NC];
  double total = 0.0;
#pragma unroll
  for (int k = 0; k < NC; k++) {
    const int c = (k * lanes + in_row) * 8, left = count(k);
    s[k] = WHOLE ? widen<DT>(in[k]) : take8<DT>(in[k], left, width);
    if (g.residual) {
      s[k] += WHOLE ? widen<DT>(add[k]) : take8<DT>(add[k], left, width);
      // the stored, rounded sum is what is normalised
      s[k] = __builtin_convertvector(__builtin_convertvector(s[k], typename Elem<DT>::vec), f32x8);
      if (live) store8<DT, NT>(g.sum + row * g.sum_stride + c, left, s[k]);
    }
#pragma unroll
    for (int i = 0; i < 8; i++) total += (double)s[k][i];
  }
  const double m = sum_row(total, lanes, 0, slots[0]) * g.inv_width;
  // differences from the mean: with codes they stay in fp64 for the output
  constexpr int kHeld = CODES ? NC : 1;
  double held[kHeld][8];
  double sq = 0.0;
#pragma unroll
  for (int k = 0; k < NC; k++) {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const double d = (double)s[k][i] - m;
      if (WHOLE || i < count(k)) sq = __builtin_fma(d, d, sq);
      if (CODES) held[CODES ? k : 0][i] = d;
    }
  }
  const double variance = sum_row(sq, lanes, 0, slots[1]) * g.inv_width;
  const double root = inverse_root(variance + (double)g.eps);
  const float r = (float)root;
  // the mean in two parts: a difference from it is off by two roundings of itself
  const float m_high = (float)m, m_low = (float)(m - (double)m_high);
  if (live && in_row == 0) {
    g.mean[row] = m_high;
    g.rstd[row] = r;
  }
  if constexpr (!CODES) {
    // As a multiplication of s in a branch of its own, eight chunks a thread spill all over: 4096 x
    // 65536 bf16 4250 us for 730; with fp16 taking the second of the ways below too, 820.
    const bool far = far_apart<DT>(r);
    const float part = far ? 0.25f : 1.0f, high = m_high * part, low = m_low * part;
    const float inverse = far ? (float)(root * 4.0) : r;
#pragma unroll
    for (int k = 0; k < NC; k++) {
      const int c = (k * lanes + in_row) * 8, left = count(k);
      if (!live || left <= 0 || !g.y) continue;
      const f32x8 w = load8<DT>(g.weight + c, left);
      const f32x8 b = g.bias ? load8<DT>(g.bias + c, left) : f32x8{};
      f32x8 v;
      if (DT == ZS_F16)
        v = ((s[k] - m_high) - m_low) * r * w + b;
      else
        v = (__builtin_elementwise_fma(s[k], (f32x8)part, (f32x8)(-high)) - low) * inverse * w + b;
      store8<DT, NT>(g.y + row * g.y_stride + c, left, v);
    }
  } else {
    const int group_lanes = g.group_lanes, groups = (width + group_lanes * 8 - 1) / (group_lanes * 8);
    // the scales that fill a span of the 4-bit form up: 15 at most, one a lane
    if (g.code == ZS_E2M1 && live && groups + in_row < (groups + 15) / 16 * 16)
      g.scales[scale4_at(row, groups + in_row, g.rows)] = 127;
#pragma unroll
    for (int k = 0; k < NC; k++) {
      const int chunk = k * lanes + in_row, c = chunk * 8, left = count(k);
      f32x8 v = {};
      double q[8] = {};
      typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
      u16x2 nearest = {0xffff, 0xffff};  // the least of the outputs' low halves
      if (WHOLE || left > 0) {
        const f32x8 w = load8<DT>(g.weight + c, left);
        const f32x8 b = g.bias ? load8<DT>(g.bias + c, left) : f32x8{};
#pragma unroll
        for (int i = 0; i < 8; i++) {
          q[i] = __builtin_fma(held[k][i] * root, (double)w[i], (double)b[i]);
          v[i] = (float)q[i];
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          nearest = __builtin_elementwise_min(nearest, __builtin_bit_cast(u16x2, __builtin_amdgcn_perm(
              __float_as_uint(v[i + 1]), __float_as_uint(v[i]), 0x05040100)));
        if (live && g.y) store8<DT, NT>(g.y + row * g.y_stride + c, left, v);
      }
      // Ties of codes, and borders of scales, have sixteen zeros at least at their end (where
      // they are normal in fp32).  An output that fp32 rounds to such a value may lie to either
      // side.
      float amax = amax_lanes(v, group_lanes);
      // the same for all lanes of a group
      const bool border = (__float_as_uint(amax) & 0xffffu) == 0 || amax < 0x1p-90f;
      if (border || nearest[0] == 0 || nearest[1] == 0) {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = side_of(q[i]);
      }
      if (border) amax = amax_lanes(v, group_lanes);
      const uint32_t byte = scale_byte_of(g.code, amax);
      // the scaling is exact but far below the group's largest, where all that matters is the side
      v *= scale_inverse(byte == 255u ? 127u : byte);
      if (g.code == ZS_E2M1) {
        const uint32_t word = byte == 255u ? 0u : encode4(v, 1.0f);
        if (live && c < groups * 32) {  // zeros behind the row's end
          *(uint32_t*)(g.codes + row * groups * 16 + chunk * 4) = word;
          if (chunk % 4 == 0) g.scales[scale4_at(row, chunk / 4, g.rows)] = (uint8_t)byte;
        }
      } else {
        u32x2 word;
        if (g.code == ZS_E4M3)
          word = encode8<ZS_E4M3>(v);
        else
          word = encode8<ZS_E5M2>(v);
        if (byte == 255u) word = u32x2{0, 0};
        if (live && left > 0) {
          store_codes<NT>(g.codes + row * width + c, left, word);
          if ((chunk & (group_lanes - 1)) == 0) g.scales[row * groups + chunk / group_lanes] = (uint8_t)byte;
        }
      }
    }
  }
}

template <int DT, bool NT, int NC, int T, bool CODES>
__global__ __launch_bounds__(T) void layer_norm_kernel(RowArgs<DT> g) {
  __shared__ double slots[2][16];
  if (g.width == g.lanes * NC * 8)
    layer_norm_rows<DT, NT, NC, CODES, true>(g, slots);
  else
    layer_norm_rows<DT, NT, NC, CODES, false>(g, slots);
}

// The first n of eight values, zeros for the others.
__device__ __forceinline__ f32x8 first_of(f32x8 x, int n) {
#pragma unroll
  for (int i = 0; i < 8; i++) x[i] = i < n ? x[i] : 0.0f;
  return x;
}

// h = (s - mean) rstd of a row; where it is far apart, the differences in quarters.
template <int DT>
struct Scaled {
  float part, mean, rstd;  // of the differences, and the others accordingly
  __device__ __forceinline__ Scaled(float m, float r) {
    const bool far = far_apart<DT>(r);
    part = far ? 0.25f : 1.0f;
    mean = m * part;
    rstd = far ? r * 4.0f : r;
  }
  __device__ __forceinline__ f32x8 operator()(f32x8 s) const {
#pragma unroll
    for (int i = 0; i < 8; i++) s[i] = __builtin_fmaf(s[i], part, -mean) * rstd;
    return s;
  }
};

// The chunks of a row that the backward pass reads.
template <int DT, int NC>
struct GradRow {
  Chunk<DT> s[NC], dy[NC], ds[NC];
  float mean, rstd;
};

constexpr int kGradThreads = 512;

template <int DT, bool NT, int NC>
__global__ __launch_bounds__(kGradThreads) void layer_norm_grad_kernel(
    const elem_t<DT>* dy, int64_t dy_stride, const elem_t<DT>* sum, int64_t sum_stride,
    const elem_t<DT>* __restrict__ weight, const float* __restrict__ mean,
    const float* __restrict__ rstd, const elem_t<DT>* ds, int64_t ds_stride, elem_t<DT>* dx,
    int64_t dx_stride, float* __restrict__ parts, int64_t part_stride, int64_t rows, int32_t width,
    int lanes, int rows_per_block) {
  __shared__ f32x2 slots[2][kGradThreads / 64];
  __shared__ __attribute__((aligned(16))) float all[kGradThreads * 8];
  const int in_row = threadIdx.x & (lanes - 1), sub = threadIdx.x / lanes;
  const int64_t step = (int64_t)gridDim.x * rows_per_block;
  const float inv_width = 1.0f / (float)width;
  const bool whole = width == lanes * NC * 8;
  f32x8 w[NC], dw[NC], db[NC];
#pragma unroll
  for (int k = 0; k < NC; k++) {
    const int c = (k * lanes + in_row) * 8;
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
      const int c = (k * lanes + in_row) * 8;
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
    const Scaled<DT> scaled(now.mean, now.rstd);
    auto take = [&](const Chunk<DT>& x, int k) {  // zeros behind the row's end, and for no row
      if (whole && row < rows) return widen<DT>(x);
      const int left = row < rows ? width - (k * lanes + in_row) * 8 : 0;
      return take8<DT>(x, left, width);
    };
#pragma unroll
    for (int k = 0; k < NC; k++) {
      h[k] = scaled(take(now.s[k], k));
      // zeros behind the row's end and for no row: -mean rstd, which may be infinite, is not one
      if (!whole || row >= rows) h[k] = first_of(h[k], row < rows ? width - (k * lanes + in_row) * 8 : 0);
      g[k] = take(now.dy[k], k);
      dw[k] += g[k] * h[k];
      db[k] += g[k];
      g[k] *= w[k];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        dot[0] += g[k][i];
        dot[1] += g[k][i] * h[k][i];
      }
    }
    const f32x2 means = sum_row(dot, lanes, sub * lanes / 64, slots[turn]) * inv_width;
#pragma unroll
    for (int k = 0; k < NC; k++) {
      const int c = (k * lanes + in_row) * 8, left = row < rows ? width - c : 0;
      const f32x8 v = (g[k] - means[0] - h[k] * means[1]) * now.rstd + take(now.ds[k], k);
      store8<DT, NT>(dx + row * dx_stride + c, left, v);
    }
  }
  float* part = parts + blockIdx.x * 2 * part_stride;
#pragma unroll
  for (int q = 0; q < 2 * NC; q++) {
    const int k = q >> 1, c = (k * lanes + in_row) * 8;
    f32x8 x = q & 1 ? db[k] : dw[k];
    if (rows_per_block > 1) {  // the workgroup's rows' parts are added here, in order
      if (q) __syncthreads();
      store8<ZS_F32>(all + threadIdx.x * 8, 8, x);
      __syncthreads();
      if (sub == 0)
        for (int i = 1; i < rows_per_block; i++) x += load8<ZS_F32>(all + (i * lanes + in_row) * 8, 8);
    }
    if (sub == 0 && c < width) store8<ZS_F32>(part + (q & 1) * part_stride + c, 8, x);
  }
}

// Wide rows, first: mean g and mean(g h) of each row.
template <int DT>
__global__ __launch_bounds__(1024) void wide_means_kernel(
    const elem_t<DT>* __restrict__ dy, int64_t dy_stride, const elem_t<DT>* __restrict__ sum,
    int64_t sum_stride, const elem_t<DT>* __restrict__ weight, const float* __restrict__ mean,
    const float* __restrict__ rstd, f32x2* __restrict__ means, int64_t width) {
  __shared__ f32x2 slots[16];
  const int64_t row = blockIdx.x;
  const Scaled<DT> scaled(mean[row], rstd[row]);
  f32x2 dot = {};
  for (int64_t c = threadIdx.x * 8; c < width; c += 1024 * 8) {
    const int64_t left = width - c;
    const Chunk<DT> a = load_row<DT>(sum + row * sum_stride, c, width);
    const Chunk<DT> b = load_row<DT>(dy + row * dy_stride, c, width);
    const f32x8 h = first_of(scaled(take8<DT>(a, left, width)), (int)(left < 8 ? left : 8));
    const f32x8 g = take8<DT>(b, left, width) * load8<DT>(weight + c, left);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      dot[0] += g[i];
      dot[1] += g[i] * h[i];
    }
  }
  const float inv_width = 1.0f / (float)width;
  const f32x2 both = sum_row(dot, 1024, 0, slots) * inv_width;
  if (threadIdx.x == 0) means[row] = both;
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
    const float r = rstd[row];
    const f32x2 both = means[row];
    const f32x8 h = Scaled<DT>(mean[row], r)(take8<DT>(a, left, width));
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

// Calls f with whether a call's data are streamed; fp32's never are.
template <int DT, typename F>
void with_streaming(bool nt, F f) {
  if constexpr (DT == ZS_F32)
    f(std::integral_constant<bool, false>());
  else
    with_bool(nt, f);
}

// How the backward pass spreads rows of up to 8192 columns: as the forward, but always over
// workgroups of 512, which add their rows' parts of dw and db, so that there are few parts (3001
// x 1001: 17.7 us for 19.9 with two thousand, a call's launches and Python included).
Shape grad_shape(int64_t width) {
  const Shape s = shape(width);
  return {s.lanes, s.nc, kGradThreads};
}

// Workgroups of the backward pass, each with a part of dw and db: two on each compute unit.  Of
// wide rows: slices of them for each strip.
int64_t grad_blocks(int64_t rows, int64_t width) {
  if (width > kHeldWidth) {
    const int64_t strips = (width + kStrip - 1) / kStrip, slices = 2048 / strips;
    return rows < slices ? rows : slices;
  }
  const Shape s = grad_shape(width);
  const int per = s.threads / s.lanes;
  const int64_t need = (rows + per - 1) / per;
  return need < 512 ? need : 512;
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
    constexpr int kDt = decltype(DT)::value;
    using E = elem_t<kDt>;
    const RowArgs<kDt> g{(const E*)x, (const E*)residual, (const E*)weight, (const E*)bias, (E*)sum, (E*)y,
                         x_stride, residual_stride, sum_stride, y_stride, (uint8_t*)codes,
                         (uint8_t*)scales, mean, rstd, rows, (int32_t)width, s.lanes, per, code,
                         group_lanes, eps, 1.0 / (double)width};
    with_streaming<kDt>(nt, [&](auto NT) {
      with_bool(codes != nullptr, [&](auto CODES) {
        with_shape(s, [&](auto NC, auto T) {
          layer_norm_kernel<kDt, decltype(NT)::value, decltype(NC)::value, decltype(T)::value,
                            decltype(CODES)::value>
              <<<dim3((uint32_t)blocks), dim3(s.threads), 0, (hipStream_t)stream>>>(g);
        });
      });
    });
  });
  return launched(who);
}

extern "C" size_t zs_layer_norm_backward_bytes(int64_t rows, int64_t width) {
  if (rows < 0 || rows > 0x7fffffff || width < 1 || width > kMaxWidth) return 0;
  const size_t parts = (size_t)grad_blocks(rows, width);
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
  const Shape s = grad_shape(width);
  const int per = s.threads / s.lanes;
  const int64_t blocks = grad_blocks(rows, width);
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
      with_streaming<kDt>(nt, [&](auto NT) {
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
        auto go = [&](auto NC) {
          layer_norm_grad_kernel<kDt, kNt, decltype(NC)::value>
              <<<dim3((uint32_t)blocks), dim3(kGradThreads), 0, (hipStream_t)stream>>>(
                  (const E*)dy, dy_stride, (const E*)sum, sum_stride, (const E*)weight, mean, rstd,
                  (const E*)grad_sum, grad_sum_stride, (E*)grad_x, grad_x_stride, parts, stride,
                  rows, (int32_t)width, s.lanes, per);
        };
        if (s.nc == 1)
          go(std::integral_constant<int, 1>());
        else
          go(std::integral_constant<int, 2>());
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
