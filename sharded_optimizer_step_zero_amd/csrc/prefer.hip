// prefer.hip -- the preference loss of pairs of packed sequences, and its gradient.
//
// With l_t the policy's -log p of token t and r_t the reference's (0 without one), a sequence
// has a = -sum (l_t - r_t) over its tokens that count, or the mean of them; a pair has m = beta
// (a_chosen - a_rejected) - margin and
//   sigmoid   L = -(1-s) log sigma(m) - s log sigma(-m)
//   hinge     L = max(0, 1 - m)
//   squared   L = (m - 1/2)^2 / beta^2
// The gradient of sum_p grad_p L_p by l_t is -+ beta L'(m) grad_p (over the length for means) for
// the tokens of the chosen and of the rejected.  A token without probability (l or r infinite) makes
// the margin infinite, where these have their limits: 0 of the hinge and of the sigmoid's side
// that is certain.
//
// Bound by latency up to some 100 thousand tokens, by HBM beyond.  Forward: half a workgroup a
// sequence, sums in fp64 in a fixed order, the loss by its last step; few long sequences are
// divided over workgroups, and a second kernel adds the parts.  Backward: a thread has four
// neighbouring tokens and looks for their sequence among the offsets, so the work is even
// whatever the lengths and every token is written once, those of no sequence too (zeros).
// Measured: 4 pairs of 1600 tokens in all 3.6 + 4.7 us, 256 pairs of a million tokens, with a mask, 6
// us (0.9 TB/s) + 8 (every thread's search is nine loads of offsets, each behind the one before); a
// launch alone takes 3.
#include <algorithm>

#include "ops.h"

namespace zs {
namespace ops {
namespace {

constexpr int64_t kMaxPairs = 1ll << 22;
constexpr int64_t kMaxTokens = (1ll << 31) - 1;

struct PreferArgs {
  const float *loss, *ref;
  const void* offsets;
  const uint8_t* mask;
  int64_t tokens, pairs;
  int32_t offset_bytes, kind, average;
  float beta, margin, smoothing;
  float *loss_out, *rewards, *margins;
  int32_t* lengths;
};

// Offset i, brought within the tokens: a wrong one must not lead out of the buffers.
__device__ __forceinline__ int64_t offset_of(const PreferArgs& g, int64_t i) {
  const int64_t o = g.offset_bytes == 8 ? ((const int64_t*)g.offsets)[i] : ((const int32_t*)g.offsets)[i];
  return o < 0 ? 0 : o > g.tokens ? g.tokens : o;
}

// A sum of differences and how many they are.
struct Part {
  double sum;
  int64_t n;
};

// Slice s of S of sequence `seq`, over 256 threads of which this is the `thread`-th; the whole
// in thread 0 of each wave.
__device__ __forceinline__ Part slice_sum(const PreferArgs& g, int64_t seq, int64_t s, int64_t S,
                                          int thread) {
  const int64_t from = offset_of(g, seq), to = offset_of(g, seq + 1);
  const int64_t len = to > from ? to - from : 0;
  const int64_t begin = from + len * s / S, end = from + len * (s + 1) / S;
  Part p = {0.0, 0};
#pragma unroll 4
  for (int64_t t = begin + thread; t < end; t += 256) {
    const bool counts = !g.mask || g.mask[t];
    const double d = (double)g.loss[t] - (g.ref ? (double)g.ref[t] : 0.0);
    p.sum += counts ? d : 0.0;
    p.n += counts;
  }
  for (int d = 1; d < 64; d <<= 1) {
    p.sum += __shfl_xor(p.sum, d, 64);
    p.n += __shfl_xor((int)p.n, d, 64);
  }
  return p;
}

__device__ __forceinline__ double softplus(double x) {  // log(1 + e^x)
  return (x > 0.0 ? x : 0.0) + log1p(exp(-fabs(x)));
}

__device__ __forceinline__ void finish_pair(const PreferArgs& g, int64_t pair, Part chosen,
                                            Part rejected) {
  double a[2];
  const Part p[2] = {chosen, rejected};
#pragma unroll
  for (int h = 0; h < 2; h++) {
    a[h] = -p[h].sum * (double)g.beta;
    if (g.average) a[h] /= (double)(p[h].n > 0 ? p[h].n : 1);
    g.rewards[pair * 2 + h] = (float)a[h];
    g.lengths[pair * 2 + h] = (int32_t)p[h].n;
  }
  const double m = a[0] - a[1] - (double)g.margin, s = g.smoothing;
  double loss;
  if (g.kind == ZS_SIGMOID)
    loss = (1.0 - s) * softplus(-m) + (s > 0.0 ? s * softplus(m) : 0.0);  // not 0 times infinity
  else if (g.kind == ZS_HINGE)
    loss = m < 1.0 ? 1.0 - m : m >= 1.0 ? 0.0 : m;  // NaN stays NaN
  else
    loss = (m - 0.5) * (m - 0.5) / ((double)g.beta * (double)g.beta);
  // The slope is taken from the margin as it is returned, in fp32: that moves it by no more than
  // rounding every token's difference to fp32 once would.  The hinge has a step in it: a margin
  // below 1 stays below.
  const float held = (float)m;
  g.margins[pair] = g.kind == ZS_HINGE && m < 1.0 && held >= 1.0f ? 0x1.fffffep-1f : held;
  g.loss_out[pair] = (float)loss;
}

// A pair a workgroup: waves 0 to 3 have the chosen sequence, 4 to 7 the rejected.
__global__ __launch_bounds__(512) void pair_kernel(PreferArgs g) {
  __shared__ Part slots[8];
  const int64_t pair = blockIdx.x;
  const int half = threadIdx.x >> 8;
  const Part p = slice_sum(g, pair * 2 + half, 0, 1, threadIdx.x & 255);
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = p;
  __syncthreads();
  if (threadIdx.x) return;
  Part both[2] = {{0.0, 0}, {0.0, 0}};
  for (int w = 0; w < 8; w++) {
    both[w >> 2].sum += slots[w].sum;
    both[w >> 2].n += slots[w].n;
  }
  finish_pair(g, pair, both[0], both[1]);
}

// Slices: blockIdx.x of gridDim.x of sequence blockIdx.y.
__global__ __launch_bounds__(256) void slice_kernel(PreferArgs g, Part* __restrict__ parts) {
  __shared__ Part slots[4];
  const Part p = slice_sum(g, blockIdx.y, blockIdx.x, gridDim.x, threadIdx.x);
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = p;
  __syncthreads();
  if (threadIdx.x) return;
  Part all = slots[0];
  for (int w = 1; w < 4; w++) {
    all.sum += slots[w].sum;
    all.n += slots[w].n;
  }
  parts[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = all;
}

__global__ __launch_bounds__(256) void join_kernel(PreferArgs g, const Part* __restrict__ parts,
                                                   int64_t slices) {
  const int64_t pair = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (pair >= g.pairs) return;
  Part both[2] = {{0.0, 0}, {0.0, 0}};
  for (int h = 0; h < 2; h++)
    for (int64_t s = 0; s < slices; s++) {
      const Part p = parts[(pair * 2 + h) * slices + s];
      both[h].sum += p.sum;
      both[h].n += p.n;
    }
  finish_pair(g, pair, both[0], both[1]);
}

// Slices of a sequence: until the card has some 512 workgroups, each slice 4096 tokens on the
// average or more.  us undivided and divided, in a graph (pairs x tokens a sequence): 4 x 8192 7.8 and
// 6.9, 4 x 32768 21 and 7.7, 64 x 16384 12.5 and 7.7.  Slices of 2048 take 5.8 for 5.5 at 4 x 4096, 6.0
// for 6.9 at 4 x 8192 and 15 for 11 at 1 x 131072; 256 workgroups 15 for 11 at 64 x 32768, 1024 32 for
// 21 at 4 x 524288.
int64_t slices_of(int64_t tokens, int64_t pairs) {
  const int64_t wanted = 256 / std::max<int64_t>(pairs, 1), most = tokens / (std::max<int64_t>(pairs, 1) * 2) / 4096;
  return std::max<int64_t>(1, std::min(wanted, most));
}

// Four tokens a thread.
__global__ __launch_bounds__(256) void prefer_grad_kernel(PreferArgs g,
                                                          const float* __restrict__ grad_loss,
                                                          float* __restrict__ grad) {
  const int64_t t0 = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (t0 >= g.tokens) return;
  const int64_t last = g.pairs * 2;
  // the last sequence that begins at or before t (offsets do not fall), of those from `low` on:
  // -1 before the first, `last` behind all of them
  auto find = [&](int64_t t, int64_t low) {
    int64_t high = last;
    if (offset_of(g, high) <= t) return high;
    while (high - low > 1) {
      const int64_t mid = (low + high) >> 1;
      if (offset_of(g, mid) <= t)
        low = mid;
      else
        high = mid;
    }
    return low;
  };
  auto end_of = [&](int64_t s) { return s < last ? offset_of(g, s + 1) : g.tokens; };
  int64_t seq = find(t0, -1), end = end_of(seq);
  auto factor = [&](int64_t s) {
    if (s < 0 || s >= last) return 0.0f;
    const int64_t pair = s >> 1;
    const double m = g.margins[pair], smooth = g.smoothing;
    double slope;
    if (g.kind == ZS_SIGMOID)
      slope = smooth - 1.0 / (1.0 + exp(m));  // -(1-s) sigma(-m) + s sigma(m)
    else if (g.kind == ZS_HINGE)
      slope = m < 1.0 ? -1.0 : m >= 1.0 ? 0.0 : m;
    else
      slope = 2.0 * (m - 0.5) / ((double)g.beta * (double)g.beta);
    slope *= (double)g.beta * (double)grad_loss[pair];
    if (g.average) {
      const int32_t n = g.lengths[s];
      slope /= (double)(n > 0 ? n : 1);
    }
    return (float)(s & 1 ? slope : -slope);
  };
  float f = factor(seq);
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int64_t t = t0 + i;
    if (t >= g.tokens) return;
    if (t >= end && seq < last) {  // the next one, or the one behind any number of empty ones
      end = end_of(++seq);
      if (t >= end && seq < last) end = end_of(seq = find(t, seq));
      f = factor(seq);
    }
    grad[t] = g.mask && !g.mask[t] ? 0.0f : f;
  }
}

int check(const char* who, const PreferArgs& g) {
  if (g.tokens < 0 || g.tokens > kMaxTokens || g.pairs < 0 || g.pairs > kMaxPairs)
    return fail(who, "a size is out of range");
  if (g.offset_bytes != 4 && g.offset_bytes != 8) return fail(who, "offsets have 4 or 8 bytes");
  if (g.kind != ZS_SIGMOID && g.kind != ZS_HINGE && g.kind != ZS_SQUARED)
    return fail(who, "unknown kind of loss");
  if (!(g.beta > 0.0f) || !__builtin_isfinite(g.beta)) return fail(who, "beta must be finite and above 0");
  if (!__builtin_isfinite(g.margin)) return fail(who, "the margin must be finite");
  if (!(g.smoothing >= 0.0f && g.smoothing <= 0.5f)) return fail(who, "smoothing must be in 0..0.5");
  if (g.smoothing != 0.0f && g.kind != ZS_SIGMOID) return fail(who, "smoothing goes with the sigmoid loss");
  if (!g.offsets || !al(g.offsets, (size_t)g.offset_bytes))
    return fail(who, "the offsets are NULL or not aligned to their elements");
  return ZS_OK;
}

}  // namespace
}  // namespace ops
}  // namespace zs

using namespace zs::ops;

extern "C" size_t zs_prefer_workspace_bytes(int64_t tokens, int64_t pairs) {
  if (tokens < 0 || tokens > kMaxTokens || pairs < 0 || pairs > kMaxPairs) return 0;
  const int64_t slices = slices_of(tokens, pairs);
  return (slices > 1 ? up256((size_t)(pairs * 2 * slices) * sizeof(Part)) : 0) + 256;
}

extern "C" int zs_prefer_forward(const float* loss, const float* ref_loss, const void* offsets,
                                 const void* mask, float* pair_loss, float* rewards,
                                 float* margins, int32_t* lengths, int64_t tokens, int64_t pairs,
                                 float beta, float margin, float smoothing, int32_t kind,
                                 int32_t average, int32_t offset_bytes, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const char* who = "zs_prefer_forward";
  PreferArgs g{loss, ref_loss, offsets, (const uint8_t*)mask, tokens, pairs, offset_bytes, kind,
               average != 0, beta, margin, smoothing, pair_loss, rewards, margins, lengths};
  if (int rc = check(who, g)) return rc;
  if (pairs == 0) return ZS_OK;
  if ((tokens && !loss) || !pair_loss || !rewards || !margins || !lengths) return fail(who, "NULL buffer");
  if (!al(loss, 4) || !al(ref_loss, 4) || !al(pair_loss, 4) || !al(rewards, 4) || !al(margins, 4) ||
      !al(lengths, 4))
    return fail(who, "a buffer is not aligned to its elements");
  const int64_t slices = slices_of(tokens, pairs);
  if (slices > 1 && (!workspace || !al(workspace, 256)))
    return fail(who, "the workspace is NULL or not 256-byte aligned");
  if (workspace_bytes < zs_prefer_workspace_bytes(tokens, pairs)) return fail(who, "the workspace is too small");
  const hipStream_t st = (hipStream_t)stream;
  if (slices == 1) {
    pair_kernel<<<dim3((uint32_t)pairs), dim3(512), 0, st>>>(g);
    return launched(who);
  }
  slice_kernel<<<dim3((uint32_t)slices, (uint32_t)(pairs * 2)), dim3(256), 0, st>>>(g, (Part*)workspace);
  if (int rc = launched(who)) return rc;
  join_kernel<<<dim3((uint32_t)((pairs + 255) / 256)), dim3(256), 0, st>>>(g, (const Part*)workspace, slices);
  return launched(who);
}

extern "C" int zs_prefer_backward(const float* margins, const int32_t* lengths,
                                  const void* offsets, const void* mask, const float* grad_loss,
                                  float* grad, int64_t tokens, int64_t pairs, float beta,
                                  float smoothing, int32_t kind, int32_t average,
                                  int32_t offset_bytes, void* stream) {
  const char* who = "zs_prefer_backward";
  PreferArgs g{nullptr, nullptr, offsets, (const uint8_t*)mask, tokens, pairs, offset_bytes, kind,
               average != 0, beta, 0.0f, smoothing, nullptr, nullptr, (float*)margins, (int32_t*)lengths};
  if (int rc = check(who, g)) return rc;
  if (tokens == 0) return ZS_OK;
  if (!grad || (pairs && (!margins || !lengths || !grad_loss))) return fail(who, "NULL buffer");
  if (!al(margins, 4) || !al(lengths, 4) || !al(grad_loss, 4) || !al(grad, 4))
    return fail(who, "a buffer is not aligned to its elements");
  prefer_grad_kernel<<<dim3((uint32_t)((tokens + 1023) / 1024)), dim3(256), 0, (hipStream_t)stream>>>(
      g, grad_loss, grad);
  return launched(who);
}
