// act8.hip -- activations held in 8 bits: packing, unpacking, and the gated unit
// that keeps its input so and takes its gradient from it.
//
// All four are one pass over their arrays and bound by HBM: a lane takes 8
// neighbouring elements (16 bytes of a 16-bit type, 8 bytes of codes), a group's
// maximum is a few shuffles among neighbouring lanes.  The scales are powers of
// two, so scaling is exact and a code is the input rounded once.  The gated unit
// reads gate and up once for its output and their codes.  The backward pass needs
// 2 bytes of checkpoint a pair where the 16-bit input takes 4, and gives the
// unit's output again so that it need not be kept either.  Measured, bf16: forward at
// 8192 x 11008 128 us for 722 MB (5.6 TB/s), backward at 4096 x 28672 189 us for 1.18 GB
// (6.2 TB/s); with plain loads and stores 136 and 199.
#include "ops.h"

namespace zs {
namespace ops {
namespace {

constexpr int64_t kMaxWidth = 1 << 20;
constexpr int64_t kMaxBlocks = 0x7fffff;

// A row takes `lanes` (16..256, a power of two) threads a block; wider rows take
// several blocks.
struct Place {
  int64_t row, chunk;
  bool live;
};
struct Spread {
  int lanes_log2;
  uint32_t per_row;  // blocks a row
  int64_t blocks;
};
Spread spread(int64_t rows, int64_t width) {
  const int64_t chunks = (width + 7) / 8;
  Spread s{4, 1, 0};
  while (s.lanes_log2 < 8 && (1ll << s.lanes_log2) < chunks) s.lanes_log2++;
  s.per_row = (uint32_t)((chunks + (1 << s.lanes_log2) - 1) >> s.lanes_log2);
  const int64_t row_blocks = (rows + (256 >> s.lanes_log2) - 1) >> (8 - s.lanes_log2);
  s.blocks = row_blocks * s.per_row;
  return s;
}
__device__ __forceinline__ Place place(int lanes_log2, uint32_t per_row, int64_t rows,
                                       int64_t width) {
  const uint32_t rb = blockIdx.x / per_row, cb = blockIdx.x - rb * per_row;
  Place p;
  p.row = ((int64_t)rb << (8 - lanes_log2)) + (threadIdx.x >> lanes_log2);
  p.chunk = ((int64_t)cb << lanes_log2) + (threadIdx.x & ((1 << lanes_log2) - 1));
  p.live = p.row < rows && p.chunk * 8 < width;
  return p;
}

template <int DT, bool NT, int CODE>
__global__ __launch_bounds__(256) void pack_kernel(const elem_t<DT>* __restrict__ x,
                                                   int64_t x_stride, uint8_t* __restrict__ codes,
                                                   uint8_t* __restrict__ scales, int64_t rows,
                                                   int64_t width, int group_lanes, int64_t groups,
                                                   int lanes_log2, uint32_t per_row) {
  const Place p = place(lanes_log2, per_row, rows, width);
  const int64_t c = p.chunk * 8, left = width - c;
  f32x8 v = {};
  if (p.live) v = load8<DT, NT>(x + p.row * x_stride + c, left);
  uint32_t byte;
  const u32x2 w = quantise8<CODE>(v, group_amax(v, group_lanes), &byte);
  if (!p.live) return;
  store_codes<NT>(codes + p.row * width + c, left, w);
  if (p.chunk % group_lanes == 0) scales[p.row * groups + p.chunk / group_lanes] = (uint8_t)byte;
}

template <int DT, bool NT, int CODE>
__global__ __launch_bounds__(256) void unpack_kernel(const uint8_t* __restrict__ codes,
                                                     const uint8_t* __restrict__ scales,
                                                     elem_t<DT>* __restrict__ x, int64_t x_stride,
                                                     int64_t rows, int64_t width, int group_lanes,
                                                     int64_t groups, int lanes_log2,
                                                     uint32_t per_row) {
  const Place p = place(lanes_log2, per_row, rows, width);
  if (!p.live) return;
  const int64_t c = p.chunk * 8, left = width - c;
  const float s = scale_value(scales[p.row * groups + p.chunk / group_lanes]);
  const f32x8 v = decode8<CODE>(load_codes<NT>(codes + p.row * width + c, left)) * s;
  store8<DT, NT>(x + p.row * x_stride + c, left, v);
}

// The logistic function at z: s = 1 / (1 + e^-z) and q = 1 - s.  For 16-bit outputs one
// exponential of z log2 e rounded, the hardware's, and its reciprocal: off by |z| units of
// fp32 and 0 below -88, where x s is below 1e-36.
template <int DT>
struct Logistic {
  float s, q;
  __device__ __forceinline__ explicit Logistic(float z) {
    s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504f));
    q = 1.0f - s;
  }
  __device__ __forceinline__ float times(float x) const { return x * s; }
};
// For fp32 ones, held to a few units at any z.  With n the nearest whole number to |z| log2 e,
// e^-|z| is 2^-n times a power of two of at most a half, whose argument loses nothing to the
// size of z; the power 2^-n comes last, so that results keep their digits down to fp32's
// subnormals.  (For all types: glu 8192 x 11008 bf16 131 for 128 us, its gradient 4096 x 28672
// 197 for 190.)
template <>
struct Logistic<ZS_F32> {
  float s, q;
  float part;  // s without the power
  int power;
  __device__ __forceinline__ explicit Logistic(float z) {
    const bool far = __builtin_fabsf(z) > 256.0f;
    const float a = far ? 256.0f : __builtin_fabsf(z);  // NaN stays
    const float n = __builtin_rintf(a * 1.44269504f);
    const float d = __builtin_fmaf(a, 1.925963033e-8f, __builtin_fmaf(a, 1.44269502f, -n));
    const float p = __builtin_amdgcn_exp2f(-d), e = __builtin_ldexpf(p, -(int)n);
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    const bool left = z < 0.0f;
    s = left ? e * r : r;
    q = left ? r : e * r;
    part = left ? far ? 0.0f : p * r : r;  // -infinity times 0 is the formula's NaN
    power = left ? -(int)n : 0;
  }
  __device__ __forceinline__ float times(float x) const { return __builtin_ldexpf(x * part, power); }
};

// act(x), and its derivative in *slope.  The tanh form of GELU is x times the
// logistic function at 2z, z = sqrt(2/pi) (x + 0.044715 x^3).
template <int DT, int ACT>
__device__ __forceinline__ float activation(float x, float* slope) {
  if (ACT == ZS_SILU) {
    const Logistic<DT> l(x);
    *slope = l.s + x * l.s * l.q;
    return l.times(x);
  }
  const float k = 0.79788456f, xx = x * x;
  const Logistic<DT> l(2.0f * k * (x + 0.044715f * x * xx));
  const float t = l.s * l.q;
  // far out the function is flat while x^3 passes fp32: 0, not 0 * infinity
  *slope = t == 0.0f ? l.s : l.s + 2.0f * k * x * t * (1.0f + 0.134145f * xx);
  return l.times(x);
}

template <int DT, bool NT, int ACT, int CODE>
__global__ __launch_bounds__(256) void glu_kernel(
    const elem_t<DT>* __restrict__ gate_up, int64_t gu_stride, elem_t<DT>* __restrict__ out,
    int64_t out_stride, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t rows,
    int64_t width, int group_lanes, int64_t groups, int lanes_log2, uint32_t per_row) {
  const Place p = place(lanes_log2, per_row, rows, width);
  const int64_t c = p.chunk * 8, left = width - c;
  f32x8 g = {}, u = {};
  if (p.live) {
    const elem_t<DT>* src = gate_up + p.row * gu_stride + c;
    g = load8<DT, NT>(src, left);
    u = load8<DT, NT>(src + width, left);
    f32x8 o;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      float slope;
      o[i] = activation<DT, ACT>(g[i], &slope) * u[i];
    }
    store8<DT, NT>(out + p.row * out_stride + c, left, o);
  }
  if (CODE >= 0) {
    uint32_t gb, ub;
    const u32x2 gw = quantise8<CODE < 0 ? 0 : CODE>(g, group_amax(g, group_lanes), &gb);
    const u32x2 uw = quantise8<CODE < 0 ? 0 : CODE>(u, group_amax(u, group_lanes), &ub);
    if (!p.live) return;
    uint8_t* dst = codes + p.row * 2 * width + c;
    store_codes<NT>(dst, left, gw);
    store_codes<NT>(dst + width, left, uw);
    if (p.chunk % group_lanes == 0) {
      uint8_t* s = scales + p.row * 2 * groups + p.chunk / group_lanes;
      s[0] = (uint8_t)gb;
      s[groups] = (uint8_t)ub;
    }
  }
}

template <int DT, bool NT, int ACT, int CODE>
__global__ __launch_bounds__(256) void glu_grad_kernel(
    const elem_t<DT>* __restrict__ dout, int64_t dout_stride, const uint8_t* __restrict__ codes,
    const uint8_t* __restrict__ scales, elem_t<DT>* __restrict__ dgu, int64_t dgu_stride,
    elem_t<DT>* __restrict__ out, int64_t out_stride, int64_t rows, int64_t width,
    int group_lanes, int64_t groups, int lanes_log2, uint32_t per_row) {
  const Place p = place(lanes_log2, per_row, rows, width);
  if (!p.live) return;
  const int64_t c = p.chunk * 8, left = width - c;
  const uint8_t* src = codes + p.row * 2 * width + c;
  const uint8_t* sc = scales + p.row * 2 * groups + p.chunk / group_lanes;
  const f32x8 g = decode8<CODE>(load_codes<NT>(src, left)) * scale_value(sc[0]);
  const f32x8 u = decode8<CODE>(load_codes<NT>(src + width, left)) * scale_value(sc[groups]);
  const f32x8 d = load8<DT, NT>(dout + p.row * dout_stride + c, left);
  f32x8 dg, du, o;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    float slope;
    const float a = activation<DT, ACT>(g[i], &slope);
    // the slope, of about 1 at most, first: d u alone may pass fp32 where the gradient does not
    dg[i] = u[i] * slope * d[i];
    du[i] = d[i] * a;
    o[i] = a * u[i];
  }
  elem_t<DT>* dst = dgu + p.row * dgu_stride + c;
  store8<DT, NT>(dst, left, dg);
  store8<DT, NT>(dst + width, left, du);
  if (out) store8<DT, NT>(out + p.row * out_stride + c, left, o);
}

template <typename F>
void with_act(int32_t act, F f) {
  if (act == ZS_SILU)
    f(std::integral_constant<int, ZS_SILU>());
  else
    f(std::integral_constant<int, ZS_GELU>());
}

int check(const char* who, int64_t rows, int64_t width, int32_t dtype) {
  if (!good_dtype(dtype)) return fail(who, "unknown element type");
  if (rows < 0 || rows > 0x7fffffff || width < 1 || width > kMaxWidth)
    return fail(who, "a size is out of range");
  if (spread(rows, width).blocks > kMaxBlocks) return fail(who, "too many rows for one call");
  return ZS_OK;
}
int check_code(const char* who, int32_t code, int32_t group) {
  if ((code != ZS_E4M3 && code != ZS_E5M2) || !good_group(group))
    return fail(who, "the 8-bit form is e4m3 or e5m2 in groups of 32, 64 or 128");
  return ZS_OK;
}

}  // namespace
}  // namespace ops
}  // namespace zs

using namespace zs::ops;

extern "C" int zs_act8_pack(const void* x, int64_t x_stride, void* codes, void* scales,
                            int64_t rows, int64_t width, int32_t dtype, int32_t code,
                            int32_t group, void* stream) {
  const char* who = "zs_act8_pack";
  if (int rc = check(who, rows, width, dtype)) return rc;
  if (int rc = check_code(who, code, group)) return rc;
  if (x_stride < width) return fail(who, "a row stride is below width");
  if (rows == 0) return ZS_OK;
  if (!x || !codes || !scales) return fail(who, "NULL buffer");
  if (!al(x, elem_bytes(dtype))) return fail(who, "a buffer is not aligned to its elements");
  const Spread s = spread(rows, width);
  const bool nt = dtype != ZS_F32 && streams(rows * width * (1 + elem_bytes(dtype)));
  with_dtype(dtype, [&](auto DT) {
    with_bool(nt, [&](auto NT) {
      with_code(code, [&](auto CODE) {
        pack_kernel<decltype(DT)::value, decltype(NT)::value, decltype(CODE)::value>
            <<<dim3((uint32_t)s.blocks), dim3(256), 0, (hipStream_t)stream>>>(
                (const elem_t<decltype(DT)::value>*)x, x_stride, (uint8_t*)codes,
                (uint8_t*)scales, rows, width, group / 8, (width + group - 1) / group,
                s.lanes_log2, s.per_row);
      });
    });
  });
  return launched(who);
}

extern "C" int zs_act8_unpack(const void* codes, const void* scales, void* x, int64_t x_stride,
                              int64_t rows, int64_t width, int32_t dtype, int32_t code,
                              int32_t group, void* stream) {
  const char* who = "zs_act8_unpack";
  if (int rc = check(who, rows, width, dtype)) return rc;
  if (int rc = check_code(who, code, group)) return rc;
  if (x_stride < width) return fail(who, "a row stride is below width");
  if (rows == 0) return ZS_OK;
  if (!x || !codes || !scales) return fail(who, "NULL buffer");
  if (!al(x, elem_bytes(dtype))) return fail(who, "a buffer is not aligned to its elements");
  const Spread s = spread(rows, width);
  const bool nt = dtype != ZS_F32 && streams(rows * width * (1 + elem_bytes(dtype)));
  with_dtype(dtype, [&](auto DT) {
    with_bool(nt, [&](auto NT) {
      with_code(code, [&](auto CODE) {
        unpack_kernel<decltype(DT)::value, decltype(NT)::value, decltype(CODE)::value>
            <<<dim3((uint32_t)s.blocks), dim3(256), 0, (hipStream_t)stream>>>(
                (const uint8_t*)codes, (const uint8_t*)scales,
                (elem_t<decltype(DT)::value>*)x, x_stride, rows, width, group / 8,
                (width + group - 1) / group, s.lanes_log2, s.per_row);
      });
    });
  });
  return launched(who);
}

extern "C" int zs_glu_forward(const void* gate_up, int64_t gate_up_stride, void* out,
                              int64_t out_stride, void* codes, void* scales, int64_t rows,
                              int64_t width, int32_t dtype, int32_t act, int32_t code,
                              int32_t group, void* stream) {
  const char* who = "zs_glu_forward";
  if (int rc = check(who, rows, width, dtype)) return rc;
  if (act != ZS_SILU && act != ZS_GELU) return fail(who, "unknown activation");
  if ((codes == nullptr) != (scales == nullptr)) return fail(who, "codes and scales go together");
  if (codes)
    if (int rc = check_code(who, code, group)) return rc;
  if (gate_up_stride < 2 * width || out_stride < width)
    return fail(who, "a row stride is below the row's width");
  if (rows == 0) return ZS_OK;
  if (!gate_up || !out) return fail(who, "NULL buffer");
  const int eb = elem_bytes(dtype);
  if (!al(gate_up, eb) || !al(out, eb)) return fail(who, "a buffer is not aligned to its elements");
  const Spread s = spread(rows, width);
  const int g = codes ? group : 128;
  const bool nt = dtype != ZS_F32 && streams(rows * width * (3 * eb + (codes ? 2 : 0)));
  with_dtype(dtype, [&](auto DT) {
    with_bool(nt, [&](auto NT) {
      with_act(act, [&](auto ACT) {
        auto go = [&](auto CODE) {
          using E = elem_t<decltype(DT)::value>;
          glu_kernel<decltype(DT)::value, decltype(NT)::value, decltype(ACT)::value,
                     decltype(CODE)::value>
              <<<dim3((uint32_t)s.blocks), dim3(256), 0, (hipStream_t)stream>>>(
                  (const E*)gate_up, gate_up_stride, (E*)out, out_stride, (uint8_t*)codes,
                  (uint8_t*)scales, rows, width, g / 8, (width + g - 1) / g, s.lanes_log2,
                  s.per_row);
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

extern "C" int zs_glu_backward(const void* grad_out, int64_t grad_out_stride, const void* codes,
                               const void* scales, void* grad_gate_up,
                               int64_t grad_gate_up_stride, void* out, int64_t out_stride,
                               int64_t rows, int64_t width, int32_t dtype, int32_t act,
                               int32_t code, int32_t group, void* stream) {
  const char* who = "zs_glu_backward";
  if (int rc = check(who, rows, width, dtype)) return rc;
  if (act != ZS_SILU && act != ZS_GELU) return fail(who, "unknown activation");
  if (int rc = check_code(who, code, group)) return rc;
  if (grad_out_stride < width || grad_gate_up_stride < 2 * width || (out && out_stride < width))
    return fail(who, "a row stride is below the row's width");
  if (rows == 0) return ZS_OK;
  if (!grad_out || !codes || !scales || !grad_gate_up) return fail(who, "NULL buffer");
  const int eb = elem_bytes(dtype);
  if (!al(grad_out, eb) || !al(grad_gate_up, eb) || !al(out, eb))
    return fail(who, "a buffer is not aligned to its elements");
  const Spread s = spread(rows, width);
  const bool nt = dtype != ZS_F32 && streams(rows * width * ((out ? 4 : 3) * eb + 2));
  with_dtype(dtype, [&](auto DT) {
    with_bool(nt, [&](auto NT) {
      with_act(act, [&](auto ACT) {
        with_code(code, [&](auto CODE) {
          using E = elem_t<decltype(DT)::value>;
          glu_grad_kernel<decltype(DT)::value, decltype(NT)::value, decltype(ACT)::value,
                          decltype(CODE)::value>
              <<<dim3((uint32_t)s.blocks), dim3(256), 0, (hipStream_t)stream>>>(
                  (const E*)grad_out, grad_out_stride, (const uint8_t*)codes,
                  (const uint8_t*)scales, (E*)grad_gate_up, grad_gate_up_stride, (E*)out,
                  out_stride, rows, width, group / 8, (width + group - 1) / group, s.lanes_log2,
                  s.per_row);
        });
      });
    });
  });
  return launched(who);
}
