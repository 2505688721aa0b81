// clip.hip -- the gradient norm over many tensors of any 16- or 32-bit types, and their clipping
// by it: sumsq = sum of g^2, c = min(1, max / (sqrt(sumsq) + 1e-6)), out = c g.
//
// The tensors are laid out once as a table of pieces of up to 4096 elements, each with its
// addresses and types, so that ten thousand small tensors and one large matrix are the same
// kind of work and a call is two launches however many there are.  A wave takes every
// n-th piece by itself: what a small tensor takes is the way to its elements, and there are 8192
// waves on it at once.  Squares are exact in fp64 (24 bits each) and finite whatever the
// element, and are summed there in a fixed order.
//
// Bound by HBM: every gradient is read, and read again and written.  The second pass goes
// through the pieces from the last to the first, so that what the first read last is still in
// the caches.  Measured: 195 tensors of 1.3 G elements, bf16 and fp32 into bf16, 459 us (5.7 TB/s) and
// 1005; ten thousand tensors of up to 4096 and four of 4096 x 4096, bf16, 47 and 65 us (by workgroups
// in pieces of 16384: 53 and 73).
#include <algorithm>
#include <vector>

#include "ops.h"

namespace zs {
namespace ops {
namespace {

constexpr int64_t kPiece = 4096;
constexpr int64_t kMaxPieces = 1ll << 26;
constexpr int kGroups = 2048;  // workgroups of a pass over the pieces, of four waves

struct Piece {
  const void* grad;
  void* out;
  int32_t n;
  int32_t dtype, out_dtype;
  int32_t unused;
};
static_assert(sizeof(Piece) == 32, "the table's format");

// Calls f(first element, eight elements, how many of them exist) for a lane's chunks of a piece,
// whose loads come first: all eight of a whole piece, two at a time otherwise.
template <int DT, typename F>
__device__ __forceinline__ void each_chunk(const void* grad, int32_t n, F f) {
  const elem_t<DT>* p = (const elem_t<DT>*)grad;
  constexpr int kChunks = kPiece / (64 * 8);
  const int32_t at = (threadIdx.x & 63) * 8;
  if (n == kPiece) {
    constexpr int kAtOnce = DT == ZS_F32 ? kChunks / 2 : kChunks;
#pragma unroll
    for (int q = 0; q < kChunks; q += kAtOnce) {
      Chunk<DT> x[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; i++) x[i] = load_chunk<DT>(p + at + (q + i) * 512, 8);
#pragma unroll
      for (int i = 0; i < kAtOnce; i++) f(at + (q + i) * 512, widen<DT>(x[i]), 8);
    }
    return;
  }
  for (int32_t c0 = 0; c0 < n; c0 += 2 * 512) {
    Chunk<DT> x[2];
#pragma unroll
    for (int i = 0; i < 2; i++) x[i] = load_row<DT>(p, c0 + at + i * 512, n);
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int32_t c = c0 + at + i * 512;
      f(c, take8<DT>(x[i], n - c, n), n - c);
    }
  }
}

template <int DT>
__device__ __forceinline__ double piece_squares(const void* grad, int32_t n) {
  double s = 0.0;
  each_chunk<DT>(grad, n, [&](int32_t, f32x8 v, int32_t) {
#pragma unroll
    for (int i = 0; i < 8; i++) s = __builtin_fma((double)v[i], (double)v[i], s);
  });
  return s;
}

// The workgroup's sum of a value a thread, in a fixed order.
__device__ __forceinline__ double block_sum(double x, double* slots) {
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = 0.0;
  for (uint32_t i = 0; i < blockDim.x / 64; i++) s += slots[i];
  return s;
}

// A wave's first piece, the same in all of its lanes.
__device__ __forceinline__ int64_t first_piece() {
  return (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
}

__global__ __launch_bounds__(256) void squares_kernel(const Piece* __restrict__ pieces,
                                                      int64_t n_pieces,
                                                      double* __restrict__ parts) {
  __shared__ double slots[4];
  double s = 0.0;
  const int64_t step = gridDim.x * 4, first = first_piece();
  Piece next = pieces[first < n_pieces ? first : 0];  // one ahead
  for (int64_t i = first; i < n_pieces; i += step) {
    const Piece p = next;
    if (i + step < n_pieces) next = pieces[i + step];
    if (p.dtype == ZS_F32)
      s += piece_squares<ZS_F32>(p.grad, p.n);
    else if (p.dtype == ZS_BF16)
      s += piece_squares<ZS_BF16>(p.grad, p.n);
    else
      s += piece_squares<ZS_F16>(p.grad, p.n);
  }
  s = block_sum(s, slots);
  if (threadIdx.x == 0) parts[blockIdx.x] = s;
}

// The workgroups' sums, added in one order by every workgroup that needs them.
__device__ __forceinline__ double total_of(const double* parts, int32_t n, double* slots) {
  double s = 0.0;
  for (int32_t i = threadIdx.x; i < n; i += 256) s += parts[i];
  return block_sum(s, slots);
}

__global__ __launch_bounds__(256) void total_kernel(const double* __restrict__ parts, int32_t n,
                                                    double* __restrict__ sumsq) {
  __shared__ double slots[4];
  const double s = total_of(parts, n, slots);
  if (threadIdx.x == 0) *sumsq = s;
}

// A factor that may lie below fp32's normal range, where it would lose digits, in two that do not.
struct Factor {
  float first, second;
  __device__ __forceinline__ explicit Factor(double c) {
    first = c < 0x1p-120 ? 0x1p-120f : 1.0f;
    second = (float)(c < 0x1p-120 ? c * 0x1p120 : c);
  }
  __device__ __forceinline__ bool one() const { return first == 1.0f && second == 1.0f; }
};

template <int DT, int OT>
__device__ __forceinline__ void scale_piece(const Piece& p, Factor c) {
  elem_t<OT>* to = (elem_t<OT>*)p.out;
  each_chunk<DT>(p.grad, p.n, [&](int32_t k, f32x8 v, int32_t left) {
    store8<OT>(to + k, left, v * c.first * c.second);
  });
}

// The sum of squares is *sumsq, or, where that is NULL, of the `n_parts` workgroups' sums: their
// 16 KB from the L2 cost a workgroup less than a launch between the two passes.
__global__ __launch_bounds__(256) void scale_kernel(const Piece* __restrict__ pieces,
                                                    int64_t n_pieces, float max_norm,
                                                    const double* __restrict__ sumsq,
                                                    const double* __restrict__ parts, int32_t n_parts,
                                                    double* __restrict__ norm_out) {
  __shared__ double slots[4];
  const double norm = sqrt(sumsq ? *sumsq : total_of(parts, n_parts, slots));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  const double q = (double)max_norm / (norm + 1e-6);
  const Factor c(q > 1.0 ? 1.0 : q);  // NaN goes through
  const int64_t step = gridDim.x * 4, first = first_piece();
  if (first >= n_pieces) return;
  Piece next = pieces[n_pieces - 1 - first];
  for (int64_t i = first; i < n_pieces; i += step) {
    const Piece p = next;
    if (i + step < n_pieces) next = pieces[n_pieces - 1 - i - step];
    // nowhere to go, or in place and unclipped: as it is
    if (!p.out || (p.grad == p.out && c.one())) continue;
    auto go = [&](auto DT) {
      constexpr int kDt = decltype(DT)::value;
      if (p.out_dtype == ZS_F32)
        scale_piece<kDt, ZS_F32>(p, c);
      else if (p.out_dtype == ZS_BF16)
        scale_piece<kDt, ZS_BF16>(p, c);
      else
        scale_piece<kDt, ZS_F16>(p, c);
    };
    if (p.dtype == ZS_F32)
      go(std::integral_constant<int, ZS_F32>());
    else if (p.dtype == ZS_BF16)
      go(std::integral_constant<int, ZS_BF16>());
    else
      go(std::integral_constant<int, ZS_F16>());
  }
}

// Whether all elements of a tensor are one run; otherwise each row is.
bool one_run(const zs_grad_tensor& t) {
  return t.rows <= 1 || (t.grad_stride == t.width && (!t.out || t.out_stride == t.width));
}

// Calls f(grad, out, elements) for each run of adjacent elements of a tensor.
template <typename F>
void each_run(const zs_grad_tensor& t, F f) {
  const int64_t eb = elem_bytes(t.dtype), ob = elem_bytes(t.out_dtype);
  const bool whole = one_run(t);
  const int64_t runs = whole ? 1 : t.rows, n = whole ? t.rows * t.width : t.width;
  if (n == 0) return;
  for (int64_t r = 0; r < runs; r++)
    f((const uint8_t*)t.grad + r * t.grad_stride * eb,
      t.out ? (uint8_t*)t.out + r * t.out_stride * ob : nullptr, n);
}

// ZS_OK, or an error of the list; *pieces: how many it makes.
int check_list(const char* who, const zs_grad_tensor* list, int64_t n, int64_t* pieces) {
  *pieces = 0;
  if (n < 0 || (n && !list)) return fail(who, "no list");
  for (int64_t i = 0; i < n; i++) {
    const zs_grad_tensor& t = list[i];
    if (!good_dtype(t.dtype) || (t.out && !good_dtype(t.out_dtype))) return fail(who, "unknown element type");
    if (t.rows < 0 || t.width < 0 || t.rows > (1ll << 40) || t.width > (1ll << 40) ||
        (t.rows && t.width > (1ll << 40) / t.rows))
      return fail(who, "a size is out of range");
    if (t.rows > 1 && (t.grad_stride < t.width || (t.out && t.out_stride < t.width)))
      return fail(who, "a row stride is below width");
    if (t.rows && t.width && !t.grad) return fail(who, "NULL buffer");
    if (!al(t.grad, elem_bytes(t.dtype)) || (t.out && !al(t.out, elem_bytes(t.out_dtype))))
      return fail(who, "a buffer is not aligned to its elements");
    const int64_t runs = one_run(t) ? 1 : t.rows, n = one_run(t) ? t.rows * t.width : t.width;
    const int64_t each = (n + kPiece - 1) / kPiece;
    if (each && runs > kMaxPieces / each) return fail(who, "too many elements or rows");
    *pieces += runs * each;
    if (*pieces > kMaxPieces) return fail(who, "too many elements or rows");
  }
  return ZS_OK;
}

// Whether an output shares a byte with another tensor's gradient or output; a tensor's own
// gradient may be its output.
bool outputs_overlap(const zs_grad_tensor* list, int64_t n) {
  struct Range {
    uintptr_t begin, end;
    bool written;
  };
  std::vector<Range> all;
  bool any = false;
  for (int64_t i = 0; i < n; i++) {
    const zs_grad_tensor& t = list[i];
    each_run(t, [&](const void* g, void* o, int64_t m) {
      const uintptr_t a = (uintptr_t)g, b = (uintptr_t)o;
      const bool itself = o == g && t.dtype == t.out_dtype;
      if (o) all.push_back({b, b + (uintptr_t)(m * elem_bytes(t.out_dtype)), true});
      if (!itself) all.push_back({a, a + (uintptr_t)(m * elem_bytes(t.dtype)), false});
      any = any || o;
    });
  }
  if (!any) return false;
  std::sort(all.begin(), all.end(), [](const Range& a, const Range& b) { return a.begin < b.begin; });
  uintptr_t written = 0, end = 0;  // the furthest end of an output, and of anything
  for (const Range& r : all) {
    if (r.begin < written || (r.written && r.begin < end)) return true;
    end = std::max(end, r.end);
    if (r.written) written = std::max(written, r.end);
  }
  return false;
}

}  // namespace
}  // namespace ops
}  // namespace zs

using namespace zs::ops;

extern "C" int64_t zs_grads_pieces(const zs_grad_tensor* list, int64_t n) {
  int64_t pieces;
  const int rc = check_list("zs_grads_pieces", list, n, &pieces);
  return rc ? rc : pieces;
}

extern "C" int zs_grads_table(const zs_grad_tensor* list, int64_t n, void* table,
                              size_t table_bytes) {
  const char* who = "zs_grads_table";
  int64_t pieces;
  if (int rc = check_list(who, list, n, &pieces)) return rc;
  if (table_bytes < (size_t)pieces * sizeof(Piece)) return fail(who, "the table is too small");
  if (pieces == 0) return ZS_OK;
  if (!table || !al(table, 8)) return fail(who, "the table is NULL or not 8-byte aligned");
  try {
    if (outputs_overlap(list, n)) return fail(who, "an output overlaps another buffer of the list");
  } catch (...) {  // nothing leaves a C entry
    return fail(who, "no host memory to check the list with");
  }
  // whole pieces first: the last of a pass, which not every wave has, are short
  Piece* to = (Piece*)table;
  for (const bool whole : {true, false})
    for (int64_t i = 0; i < n; i++) {
      const zs_grad_tensor& t = list[i];
      each_run(t, [&](const void* g, void* o, int64_t m) {
        const int64_t rest = m / kPiece * kPiece;
        for (int64_t at = whole ? 0 : rest; at < (whole ? rest : m); at += kPiece)
          *to++ = Piece{(const uint8_t*)g + at * elem_bytes(t.dtype),
                        o ? (uint8_t*)o + at * elem_bytes(t.out_dtype) : nullptr,
                        (int32_t)std::min(kPiece, m - at), t.dtype, o ? t.out_dtype : t.dtype, 0};
      });
    }
  return ZS_OK;
}

extern "C" size_t zs_grads_workspace_bytes(int64_t pieces) {
  if (pieces < 0 || pieces > kMaxPieces) return 0;
  return up256(kGroups * 8) + 256;
}

// Enqueues the sums of squares of the workgroups, `*blocks` of them, into the workspace.
static int enqueue_squares(const char* who, const void* table, int64_t pieces, void* workspace,
                           size_t workspace_bytes, int32_t* blocks, hipStream_t stream) {
  if (!workspace || !al(workspace, 256)) return fail(who, "the workspace is NULL or not 256-byte aligned");
  if (workspace_bytes < zs_grads_workspace_bytes(pieces)) return fail(who, "the workspace is too small");
  *blocks = (int32_t)std::min<int64_t>((pieces + 3) / 4, kGroups);
  if (*blocks)
    squares_kernel<<<dim3((uint32_t)*blocks), dim3(256), 0, stream>>>((const Piece*)table, pieces,
                                                                      (double*)workspace);
  return launched(who);
}

extern "C" int zs_grads_sumsq(const void* table, int64_t pieces, double* sumsq, void* workspace,
                              size_t workspace_bytes, void* stream) {
  const char* who = "zs_grads_sumsq";
  if (pieces < 0 || pieces > kMaxPieces) return fail(who, "a size is out of range");
  if (!sumsq || (pieces && !table)) return fail(who, "NULL buffer");
  if (!al(sumsq, 8) || !al(table, 32)) return fail(who, "a buffer is not aligned to its elements");
  int32_t blocks;
  if (int rc = enqueue_squares(who, table, pieces, workspace, workspace_bytes, &blocks, (hipStream_t)stream))
    return rc;
  total_kernel<<<dim3(1), dim3(256), 0, (hipStream_t)stream>>>((const double*)workspace, blocks, sumsq);
  return launched(who);
}

extern "C" int zs_grads_clip(const void* table, int64_t pieces, float max_norm,
                             const double* sumsq, double* norm_out, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const char* who = "zs_grads_clip";
  if (pieces < 0 || pieces > kMaxPieces) return fail(who, "a size is out of range");
  if (!(max_norm > 0.0f) || !__builtin_isfinite(max_norm)) return fail(who, "max_norm must be finite and above 0");
  if (pieces && !table) return fail(who, "NULL buffer");
  if (!al(sumsq, 8) || !al(norm_out, 8) || !al(table, 32))
    return fail(who, "a buffer is not aligned to its elements");
  // one workgroup writes the norm while others may not have read the sum yet
  if (sumsq && sumsq == norm_out) return fail(who, "the sum of squares and the norm are the same buffer");
  int32_t parts = 0;
  if (!sumsq)
    if (int rc = enqueue_squares(who, table, pieces, workspace, workspace_bytes, &parts, (hipStream_t)stream))
      return rc;
  const int32_t blocks = (int32_t)std::max<int64_t>(1, std::min<int64_t>((pieces + 3) / 4, kGroups));
  scale_kernel<<<dim3((uint32_t)blocks), dim3(256), 0, (hipStream_t)stream>>>(
      (const Piece*)table, pieces, max_norm, sumsq, (const double*)workspace, parts, norm_out);
  return launched(who);
}
