// xent.hip -- softmax cross entropy of a linear head over a large vocabulary, in
// pieces of the vocabulary, without keeping the logits, and its gradient.
//
//   logits L = H W^T          [tokens, vocab], H [tokens, width], W [vocab, width]
//   lse_t = log sum_v exp L_tv,  loss_t = lse_t - L_t,target(t)
//   G_tv = grad_loss_t (exp(L_tv - lse_t) - [v = target(t)])
//   dH = G W,  dW = G^T H
//
// Forward: one matrix product whose tiles end in the maximum and the sum of
// exponentials of each token's part of the vocabulary (two floats a token and
// 128 or 32 vocabulary entries); a second kernel joins them.  Backward: pieces of the
// vocabulary; for each, the product again, its tiles ending in G (and G
// transposed), and the two products that use it.  8 * tokens * vocab * width
// operations in all, on the matrix cores: bound by their rate where there are
// tokens enough, by reading W where there are few.
//
// All three products are one kernel, C[n][m] = sum_k A[m][k] B[n][k], both
// operands with k adjacent, on 16x16x32 matrix instructions (16-bit in, fp32
// sums).  Tiles of A and B go from global memory straight into LDS, 64 elements of
// k at a time, two buffers deep; a 16-byte chunk of row r sits at chunk
// position c ^ (r & 7), so that the 16 rows a matrix instruction's operand needs do
// not meet on the same banks.  Rows past the edge and k past the width are read as
// zeros by the buffer instructions' bounds check.
#include <algorithm>

#include "ops.h"

namespace zs {
namespace ops {
namespace {

typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_ptr;

constexpr int kRsrcWord3 = 0x00020000;  // raw 32-bit buffer, gfx9 family
constexpr int BK = 64;            // k elements of one step: 128 bytes of a row
constexpr int kRowBytes = BK * 2;

constexpr int kStats = 0;   // maximum, sum of exponentials and target logit
constexpr int kGrad = 1;    // G and G transposed
constexpr int kStore = 2;   // C, rounded
constexpr int kAccum = 3;   // C in fp32, stored or added

struct GemmArgs {
  const uint16_t *a, *b;
  int64_t lda, ldb;      // row strides
  int64_t m, n, k;       // rows of A and of B, and k (a multiple of 8)
  int32_t tiles_m, tiles_n;
  int64_t k_per_split;   // a multiple of BK; the split is blockIdx.y
  // kStats, kGrad
  const void* targets;
  int32_t target_bytes;
  int64_t vocab, v0;     // A's first row is vocabulary entry v0
  float *part_max, *part_sum, *target_logit;
  const float *lse, *gloss, *gmax;
  uint16_t *g, *gt;      // G [n][ldg], G transposed [m][ldgt]
  int64_t ldg, ldgt, n_pad;  // columns of gt up to n_pad are written
  // kStore, kAccum
  uint16_t* c;
  float* acc;
  int64_t ldc, acc_split;
  int32_t add, c_wide;
};

template <int DT>
__device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c) {
  if constexpr (DT == ZS_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <int DT>
__device__ __forceinline__ uint16_t round16(float x) {
  return __builtin_bit_cast(uint16_t, (elem_t<DT>)x);
}

__device__ __forceinline__ int64_t target_of(const GemmArgs& g, int64_t t) {
  return g.target_bytes == 8 ? ((const int64_t*)g.targets)[t] : ((const int32_t*)g.targets)[t];
}

// The tile of a workgroup.  Workgroups go round the 8 dies: each die takes a
// contiguous part of the tiles, which run down a band of 8 tiles of B, so that the
// tiles at work on a die share their rows of A and B in its L2.
__device__ __forceinline__ void tile_of(const GemmArgs& g, int32_t* tm, int32_t* tn) {
  const uint32_t total = (uint32_t)g.tiles_m * (uint32_t)g.tiles_n;
  const uint32_t die = blockIdx.x & 7, per = total >> 3, extra = total & 7;
  const uint32_t id = die * per + (die < extra ? die : extra) + (blockIdx.x >> 3);
  const uint32_t band = id / ((uint32_t)g.tiles_m * 8);
  const uint32_t in = id - band * (uint32_t)g.tiles_m * 8;
  const uint32_t wide = (uint32_t)g.tiles_n - band * 8 < 8 ? (uint32_t)g.tiles_n - band * 8 : 8;
  *tm = (int32_t)(in / wide);
  *tn = (int32_t)(band * 8 + in % wide);
}

template <int DT, int BM, int BN, int WM, int WN, int EPI>
__device__ __forceinline__ void gemm(const GemmArgs& g) {
  constexpr int kThreads = WM * WN * 64;
  constexpr int kPass = kThreads / 8;  // rows that one load of all threads covers
  constexpr int PA = BM / kPass, PB = BN / kPass;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  constexpr int kTile = (BM + BN) * kRowBytes;
  static_assert(BM % kPass == 0 && BN % kPass == 0, "whole passes");
  constexpr int kOut = EPI == kGrad || EPI == kStore ? BM * BN * 2 : 0;
  constexpr int kLds = 2 * kTile > kOut ? 2 * kTile : kOut;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WN, wn = wave % WN;
  int32_t tm, tn;
  tile_of(g, &tm, &tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int64_t k_begin = blockIdx.y * g.k_per_split;
  const int64_t k_end = k_begin + g.k_per_split < g.k ? k_begin + g.k_per_split : g.k;
  const int nk = k_end > k_begin ? (int)((k_end - k_begin + BK - 1) / BK) : 0;

  // the rows of this tile that exist, from the split's first k on; a lane's
  // offsets beyond them read zeros
  const int rows_a = (int)(g.m - m0 < BM ? g.m - m0 : BM);
  const int rows_b = (int)(g.n - n0 < BN ? g.n - n0 : BN);
  const int k_len = (int)(k_end - k_begin);
  const auto ra = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(g.a + m0 * g.lda + k_begin), 0, (uint32_t)(((rows_a - 1) * g.lda + k_len) * 2),
      kRsrcWord3);
  const auto rb = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(g.b + n0 * g.ldb + k_begin), 0, (uint32_t)(((rows_b - 1) * g.ldb + k_len) * 2),
      kRsrcWord3);
  const int lr = tid >> 3;                      // row within a pass
  const int lc = (tid & 7) ^ (lr & 7);          // the 16-byte chunk that belongs there
  uint32_t off_a[PA], off_b[PB];
#pragma unroll
  for (int p = 0; p < PA; p++) off_a[p] = (uint32_t)(((lr + p * kPass) * g.lda + lc * 8) * 2);
#pragma unroll
  for (int p = 0; p < PB; p++) off_b[p] = (uint32_t)(((lr + p * kPass) * g.ldb + lc * 8) * 2);

  auto load = [&](int step, int buf) {
    // k past the end would be the next row's: such chunks go out of bounds
    const bool in = step * BK + lc * 8 < k_len;
    const uint32_t ko = (uint32_t)step * kRowBytes;
    uint8_t* base = lds + buf * kTile + wave * 8 * kRowBytes;
#pragma unroll
    for (int p = 0; p < PA; p++)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr)(base + p * kPass * kRowBytes), 16,
                                               in ? off_a[p] + ko : 0xfffffff0u, 0, 0, 0);
#pragma unroll
    for (int p = 0; p < PB; p++)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rb, (lds_ptr)(base + (BM + p * kPass) * kRowBytes), 16,
          in ? off_b[p] + ko : 0xfffffff0u, 0, 0, 0);
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int j = 0; j < FN; j++) acc[i][j] = f32x4{};

  const int row_a = wm * (BM / WM) + (lane & 15), row_b = wn * (BN / WN) + (lane & 15);
  auto compute = [&](int buf) {
    const uint8_t* ta = lds + buf * kTile;
    const uint8_t* tb = ta + BM * kRowBytes;
#pragma unroll
    for (int kk = 0; kk < BK / 32; kk++) {
      const int ch = ((kk * 4 + (lane >> 4)) ^ (lane & 7)) * 16;  // row & 7 == lane & 7
      s16x8 fa[FM], fb[FN];
#pragma unroll
      for (int i = 0; i < FM; i++)
        fa[i] = *(const s16x8*)(ta + (row_a + i * 16) * kRowBytes + ch);
#pragma unroll
      for (int j = 0; j < FN; j++)
        fb[j] = *(const s16x8*)(tb + (row_b + j * 16) * kRowBytes + ch);
#pragma unroll
      for (int i = 0; i < FM; i++)
#pragma unroll
        for (int j = 0; j < FN; j++) acc[i][j] = mfma<DT>(fa[i], fb[j], acc[i][j]);
    }
  };

  if (nk > 0) load(0, 0);
  for (int step = 0; step < nk; step++) {
    // this step's tile has arrived for every wave, and the other buffer is read out
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (step + 1 < nk) load(step + 1, (step + 1) & 1);
    compute(step & 1);
  }

  // acc[i][j][r] is C at row m0 + wm*(BM/WM) + i*16 + (lane>>4)*4 + r of A and row
  // n0 + wn*(BN/WN) + j*16 + (lane&15) of B
  const int em = wm * (BM / WM) + (lane >> 4) * 4, en = wn * (BN / WN) + (lane & 15);

  if constexpr (EPI == kStats) {
#pragma unroll
    for (int j = 0; j < FN; j++) {
      const int64_t t = n0 + en + j * 16;
      const int64_t target = t < g.n ? target_of(g, t) : -1;
      float top = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < FM; i++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
          const int64_t v = m0 + em + i * 16 + r;
          if (v < g.vocab) top = __builtin_fmaxf(top, acc[i][j][r]);
          if (v == target && v < g.vocab) g.target_logit[t] = acc[i][j][r];
        }
      top = __builtin_fmaxf(top, __shfl_xor(top, 16, 64));
      top = __builtin_fmaxf(top, __shfl_xor(top, 32, 64));
      const float from = top == -__builtin_inff() ? 0.0f : top;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < FM; i++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
          const int64_t v = m0 + em + i * 16 + r;
          if (v < g.vocab) sum += __builtin_amdgcn_exp2f((acc[i][j][r] - from) * 1.44269504f);
        }
      sum += __shfl_xor(sum, 16, 64);
      sum += __shfl_xor(sum, 32, 64);
      if (lane < 16 && t < g.n) {
        const int64_t at = (int64_t)(tm * WM + wm) * g.n + t;
        g.part_max[at] = top;
        g.part_sum[at] = sum;
      }
    }
  } else if constexpr (EPI == kAccum) {
    float* out = g.acc + blockIdx.y * g.acc_split;
#pragma unroll
    for (int j = 0; j < FN; j++) {
      const int64_t n = n0 + en + j * 16;
#pragma unroll
      for (int i = 0; i < FM; i++) {
        const int64_t m = m0 + em + i * 16;
        if (n < g.n && m < g.m) {  // rows of acc are padded to whole chunks of 4
          f32x4* p = (f32x4*)(out + n * g.ldc + m);
          *p = g.add ? *p + acc[i][j] : acc[i][j];
        }
      }
    }
  } else {
    // the tile in 16 bits in LDS, [n][m], chunks of a row swizzled by the row
    __syncthreads();
    float factor = 1.0f;
    if (EPI == kStore) factor = *g.gmax;
#pragma unroll
    for (int j = 0; j < FN; j++) {
      const int64_t t = n0 + en + j * 16;
      float lse = 0.0f, scale = 0.0f;
      int64_t target = -1;
      bool counts = false;
      if (EPI == kGrad && t < g.n) {
        target = target_of(g, t);
        counts = target >= 0 && target < g.vocab;
        lse = g.lse[t];
        const float top = *g.gmax;
        scale = top > 0.0f ? g.gloss[t] / top : g.gloss[t];
      }
#pragma unroll
      for (int i = 0; i < FM; i++) {
        uint16_t h[4];
#pragma unroll
        for (int r = 0; r < 4; r++) {
          float x = acc[i][j][r];
          if (EPI == kGrad) {
            const int64_t v = g.v0 + m0 + em + i * 16 + r;
            x = __builtin_amdgcn_exp2f((x - lse) * 1.44269504f);
            x = scale * (v == target ? x - 1.0f : x);
            if (!counts || v >= g.vocab) x = 0.0f;
          } else {
            x *= factor;
          }
          h[r] = round16<DT>(x);
        }
        const int row = en + j * 16, m = em + i * 16;
        const int ch = (m >> 3) ^ (row & (BM / 8 - 1));
        *(u32x2*)(lds + row * (BM * 2) + ch * 16 + (m & 4) * 2) =
            u32x2{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
      }
    }
    __syncthreads();
    uint16_t* out = EPI == kGrad ? g.g : g.c;
    const int64_t ldo = EPI == kGrad ? g.ldg : g.ldc;
    const bool wide = EPI == kGrad || g.c_wide;
    // G's columns reach to its stride (zeros past the vocabulary)
    const int64_t m_end = EPI == kGrad ? g.ldg : g.m;
    for (int x = tid; x < BM / 8 * BN; x += kThreads) {
      const int row = x / (BM / 8), c = x % (BM / 8);
      const int64_t n = n0 + row, m = m0 + c * 8;
      if (n >= g.n || m >= m_end) continue;
      const u32x4 w = *(const u32x4*)(lds + row * (BM * 2) + (c ^ (row & (BM / 8 - 1))) * 16);
      uint16_t* p = out + n * ldo + m;
      if (wide && m + 8 <= m_end) {
        *(u32x4*)p = w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
          if (m + i < m_end) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
      }
    }
    if (EPI == kGrad && g.gt) {
      for (int x = tid; x < BN / 8 * BM; x += kThreads) {
        const int c = x % (BN / 8), m = x / (BN / 8);
        if (m0 + m >= g.m || n0 + c * 8 >= g.n_pad) continue;
        u32x4 w = {};
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const int row = c * 8 + i;
          const uint16_t h = *(const uint16_t*)(lds + row * (BM * 2) +
                                                ((m >> 3) ^ (row & (BM / 8 - 1))) * 16 + (m & 7) * 2);
          w[i >> 1] |= (uint32_t)h << (16 * (i & 1));
        }
        *(u32x4*)(g.gt + (m0 + m) * g.ldgt + n0 + c * 8) = w;
      }
    }
  }
}

template <int DT, int BM, int BN, int WM, int WN, int EPI>
__global__ __launch_bounds__(WM* WN * 64) void gemm_kernel(GemmArgs g) {
  gemm<DT, BM, BN, WM, WN, EPI>(g);
}

// Joins a token's partial maxima and sums: 16 threads a token, each over every
// 16th part, then over the threads in order.
__global__ __launch_bounds__(256) void join_stats_kernel(
    const float* __restrict__ part_max, const float* __restrict__ part_sum,
    const float* __restrict__ target_logit, const void* __restrict__ targets,
    int32_t target_bytes, int64_t tokens, int64_t vocab, int32_t parts, float* __restrict__ loss,
    float* __restrict__ lse) {
  __shared__ float tops[16][16], sums[16][16];
  const int tt = threadIdx.x & 15, s = threadIdx.x >> 4;
  const int64_t t = (int64_t)blockIdx.x * 16 + tt;
  float top = -__builtin_inff(), sum = 0.0f;
  bool nan = false;
  if (t < tokens) {
    for (int p = s; p < parts; p += 16) top = __builtin_fmaxf(top, part_max[p * tokens + t]);
    for (int p = s; p < parts; p += 16) {
      const float m = part_max[p * tokens + t], x = part_sum[p * tokens + t];
      nan |= x != x;
      if (m != -__builtin_inff()) sum += x * __builtin_amdgcn_exp2f((m - top) * 1.44269504f);
    }
  }
  if (nan) sum = __builtin_nanf("");
  tops[s][tt] = top;
  sums[s][tt] = sum;
  __syncthreads();
  if (s != 0 || t >= tokens) return;
  top = -__builtin_inff();
  for (int i = 0; i < 16; i++) top = __builtin_fmaxf(top, tops[i][tt]);
  sum = 0.0f;
  for (int i = 0; i < 16; i++)
    if (tops[i][tt] != -__builtin_inff() || sums[i][tt] != sums[i][tt])
      sum += sums[i][tt] * __builtin_amdgcn_exp2f((tops[i][tt] - top) * 1.44269504f);
  const float l = sum == 0.0f ? -__builtin_inff() : __builtin_logf(sum) + top;
  const int64_t target =
      target_bytes == 8 ? ((const int64_t*)targets)[t] : ((const int32_t*)targets)[t];
  lse[t] = l;
  loss[t] = target >= 0 && target < vocab ? l - target_logit[t] : 0.0f;
}

// out[j][i] = in[i][j] for i < rows (0 for rows whose target does not count, and
// up to rows_pad), j < cols: 64 x 64 tiles through LDS.
__global__ __launch_bounds__(256) void transpose_kernel(const uint16_t* __restrict__ in,
                                                        int64_t in_stride, int64_t rows,
                                                        int64_t cols, uint16_t* __restrict__ out,
                                                        int64_t out_stride, int64_t rows_pad,
                                                        const void* __restrict__ targets,
                                                        int32_t target_bytes, int64_t vocab) {
  __shared__ uint16_t tile[64][66];
  const int64_t r0 = (int64_t)blockIdx.x * 64, c0 = (int64_t)blockIdx.y * 64;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int i = w; i < 64; i += 4) {
    const int64_t r = r0 + i, c = c0 + lane;
    bool in_range = r < rows && c < cols;
    if (in_range && targets) {
      const int64_t t = target_bytes == 8 ? ((const int64_t*)targets)[r] : ((const int32_t*)targets)[r];
      in_range = t >= 0 && t < vocab;
    }
    tile[i][lane] = in_range ? in[r * in_stride + c] : (uint16_t)0;
  }
  __syncthreads();
  for (int i = w; i < 64; i += 4) {
    const int64_t c = c0 + i, r = r0 + lane;
    if (c < cols && r < rows_pad) out[c * out_stride + r] = tile[lane][i];
  }
}

// Rows copied to a stride that is a multiple of 8 elements, zeros past the width.
__global__ __launch_bounds__(256) void copy_rows_kernel(const uint16_t* __restrict__ in,
                                                        int64_t in_stride, int64_t rows,
                                                        int64_t width, uint16_t* __restrict__ out,
                                                        int64_t out_stride) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t c = threadIdx.x; c < out_stride; c += 256)
      out[r * out_stride + c] = c < width ? in[r * in_stride + c] : (uint16_t)0;
}

// The largest finite |grad_loss| of the tokens that count.
__global__ __launch_bounds__(1024) void gmax_kernel(const float* __restrict__ gloss,
                                                    const void* __restrict__ targets,
                                                    int32_t target_bytes, int64_t tokens,
                                                    int64_t vocab, float* __restrict__ out) {
  __shared__ float slots[16];
  float top = 0.0f;
  for (int64_t t = threadIdx.x; t < tokens; t += 1024) {
    const int64_t v = target_bytes == 8 ? ((const int64_t*)targets)[t] : ((const int32_t*)targets)[t];
    const float x = __builtin_fabsf(gloss[t]);
    if (v >= 0 && v < vocab && x < __builtin_inff()) top = __builtin_fmaxf(top, x);
  }
  for (int d = 1; d < 64; d <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d, 64));
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 16; i++) top = __builtin_fmaxf(top, slots[i]);
    *out = top > 0.0f ? top : 1.0f;
  }
}

// grad_hidden = the splits' sums in order, times the factor, rounded.
template <int DT>
__global__ __launch_bounds__(256) void finish_kernel(const float* __restrict__ acc,
                                                     int64_t acc_stride, int64_t acc_split,
                                                     int32_t splits, const float* __restrict__ gmax,
                                                     elem_t<DT>* __restrict__ out,
                                                     int64_t out_stride, int64_t rows,
                                                     int64_t width, int32_t per_row) {
  const int64_t row = blockIdx.x / per_row;
  const int64_t c = ((int64_t)(blockIdx.x % per_row) * 256 + threadIdx.x) * 4;
  if (row >= rows || c >= width) return;
  f32x4 s = {};
  for (int i = 0; i < splits; i++) s += *(const f32x4*)(acc + i * acc_split + row * acc_stride + c);
  s *= *gmax;
  for (int i = 0; i < 4; i++)
    if (c + i < width) out[row * out_stride + c + i] = (elem_t<DT>)s[i];
}

// ---------------------------------------------------------------- host side

constexpr int64_t kMaxWidth = 65536, kMaxStride = 1 << 21, kMaxRows = 0x7fffffff - 512;
// G and its transpose of one piece together: within the 256 MB of the last-level cache
constexpr int64_t kPieceElems = 64ll << 20;
constexpr int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

bool needs_copy(const void* p, int64_t stride, int64_t width) {
  return !al(p, 16) || stride % 8 || width % 8;
}

struct Plan {
  int64_t wp;         // width in whole chunks of 8
  bool copy_h, copy_w;
  bool small;         // few tokens: tiles of 64 tokens
  int64_t bm, bn;     // tile of the products that end in tokens
  int64_t parts;      // partial statistics a token (forward)
  int64_t tp;         // tokens padded for G transposed
  int64_t piece;      // vocabulary entries a piece (backward)
  int32_t splits;     // of k in the product for grad_hidden
  size_t h, w, pmax, psum, tlogit, gmax, ht, wt, g, gt, acc, total;
};

Plan plan(const void* hidden, int64_t h_stride, const void* weight, int64_t w_stride,
          int64_t tokens, int64_t vocab, int64_t width, bool backward) {
  Plan p{};
  p.wp = up(width, 8);
  p.copy_h = needs_copy(hidden, h_stride, width);
  p.copy_w = needs_copy(weight, w_stride, width);
  p.small = tokens <= 128;
  p.bm = p.small ? 128 : 256;
  p.bn = p.small ? 64 : 256;
  p.parts = up(vocab, p.bm) / p.bm * (p.small ? 4 : 2);
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t q = at;
    at += up256((size_t)bytes);
    return q;
  };
  if (p.copy_h) p.h = take(tokens * p.wp * 2);
  if (p.copy_w) p.w = take(vocab * p.wp * 2);
  if (!backward) {
    p.pmax = take(p.parts * tokens * 4);
    p.psum = take(p.parts * tokens * 4);
    p.tlogit = take(tokens * 4);
  } else {
    p.tp = up(std::max<int64_t>(tokens, 1), 64);
    const int64_t most = std::max<int64_t>(kPieceElems / p.tp / 256 * 256, 256);
    const int64_t pieces = (vocab + most - 1) / most;
    p.piece = up((vocab + pieces - 1) / pieces, 256);
    // few tokens leave few tiles of grad_hidden: the piece's entries are divided
    // until the tiles cover the card, each part at least 512 long
    const int64_t tiles = up(width, p.bm) / p.bm * (up(std::max<int64_t>(tokens, 1), p.bn) / p.bn);
    p.splits = (int32_t)std::max<int64_t>(1, std::min<int64_t>(512 / tiles, p.piece / 512));
    p.gmax = take(4);
    p.ht = take(width * p.tp * 2);
    p.wt = take(width * p.piece * 2);
    p.g = take(tokens * p.piece * 2);
    p.gt = take(p.piece * p.tp * 2);
    p.acc = take(p.splits * tokens * p.wp * 4);
  }
  p.total = std::max<size_t>(at, 256);
  return p;
}

int check(const char* who, const void* hidden, int64_t hidden_stride, const void* weight,
          int64_t weight_stride, const void* targets, int64_t tokens, int64_t vocab,
          int64_t width, int32_t dtype, int32_t target_bytes) {
  if (dtype != ZS_BF16 && dtype != ZS_F16) return fail(who, "the element type is bf16 or fp16");
  if (tokens < 0 || tokens > kMaxRows || vocab < 1 || vocab > kMaxRows || width < 1 ||
      width > kMaxWidth)
    return fail(who, "a size is out of range");
  if (target_bytes != 4 && target_bytes != 8) return fail(who, "targets are 4 or 8 bytes");
  if (hidden_stride < width || weight_stride < width || hidden_stride > kMaxStride ||
      weight_stride > kMaxStride)
    return fail(who, "a row stride is below width or above 2^21");
  if (!weight || (tokens && (!hidden || !targets))) return fail(who, "NULL buffer");
  if (!al(hidden, 2) || !al(weight, 2) || !al(targets, target_bytes))
    return fail(who, "a buffer is not aligned to its elements");
  return ZS_OK;
}

template <int EPI>
void launch(const GemmArgs& a, bool small, int dtype, int splits, hipStream_t s) {
  const dim3 grid((uint32_t)(a.tiles_m * a.tiles_n), (uint32_t)splits);
  auto go = [&](auto DT) {
    constexpr int D = decltype(DT)::value;
    if (small)
      gemm_kernel<D, 128, 64, 4, 1, EPI><<<grid, dim3(256), 0, s>>>(a);
    else
      gemm_kernel<D, 256, 256, 2, 4, EPI><<<grid, dim3(512), 0, s>>>(a);
  };
  if (dtype == ZS_BF16)
    go(std::integral_constant<int, ZS_BF16>());
  else
    go(std::integral_constant<int, ZS_F16>());
}

// Sizes a product and checks that its grid can be launched.
bool shape(GemmArgs* a, bool small, int64_t m, int64_t n, int64_t k, int splits) {
  const int64_t bm = small ? 128 : 256, bn = small ? 64 : 256;
  a->m = m;
  a->n = n;
  a->k = k;
  const int64_t tm = up(m, bm) / bm, tn = up(n, bn) / bn;
  a->tiles_m = (int32_t)tm;
  a->tiles_n = (int32_t)tn;
  a->k_per_split = std::max<int64_t>(up((k + splits - 1) / splits, BK), BK);
  return tm * tn * 512 <= 0xffffffffll;
}

void copy_rows(const void* in, int64_t stride, int64_t rows, int64_t width, void* out,
               int64_t wp, hipStream_t s) {
  if (rows)
    copy_rows_kernel<<<dim3((uint32_t)std::min<int64_t>(rows, 4096)), dim3(256), 0, s>>>(
        (const uint16_t*)in, stride, rows, width, (uint16_t*)out, wp);
}

}  // namespace
}  // namespace ops
}  // namespace zs

using namespace zs::ops;

extern "C" size_t zs_xent_workspace_bytes(const void* hidden, int64_t hidden_stride,
                                          const void* weight, int64_t weight_stride,
                                          int64_t tokens, int64_t vocab, int64_t width,
                                          int32_t backward) {
  if (tokens < 0 || tokens > kMaxRows || vocab < 1 || vocab > kMaxRows || width < 1 ||
      width > kMaxWidth)
    return 0;
  return plan(hidden, hidden_stride, weight, weight_stride, tokens, vocab, width, backward != 0)
      .total;
}

extern "C" int zs_xent_forward(const void* hidden, int64_t hidden_stride, const void* weight,
                               int64_t weight_stride, const void* targets, float* loss,
                               float* lse, int64_t tokens, int64_t vocab, int64_t width,
                               int32_t dtype, int32_t target_bytes, void* workspace,
                               size_t workspace_bytes, void* stream) {
  const char* who = "zs_xent_forward";
  if (int rc = check(who, hidden, hidden_stride, weight, weight_stride, targets, tokens, vocab,
                     width, dtype, target_bytes))
    return rc;
  if (tokens == 0) return ZS_OK;
  if (!loss || !lse) return fail(who, "NULL buffer");
  if (!al(loss, 4) || !al(lse, 4)) return fail(who, "a buffer is not aligned to its elements");
  const Plan p = plan(hidden, hidden_stride, weight, weight_stride, tokens, vocab, width, false);
  if (!workspace || !al(workspace, 256)) return fail(who, "the workspace is NULL or not 256-byte aligned");
  if (workspace_bytes < p.total) return fail(who, "the workspace is too small");
  GemmArgs a{};
  if (!shape(&a, p.small, vocab, tokens, p.wp, 1)) return fail(who, "too many rows for one call");
  hipStream_t s = (hipStream_t)stream;
  uint8_t* ws = (uint8_t*)workspace;
  a.a = (const uint16_t*)weight;
  a.lda = weight_stride;
  a.b = (const uint16_t*)hidden;
  a.ldb = hidden_stride;
  if (p.copy_w) {
    copy_rows(weight, weight_stride, vocab, width, ws + p.w, p.wp, s);
    a.a = (const uint16_t*)(ws + p.w);
    a.lda = p.wp;
  }
  if (p.copy_h) {
    copy_rows(hidden, hidden_stride, tokens, width, ws + p.h, p.wp, s);
    a.b = (const uint16_t*)(ws + p.h);
    a.ldb = p.wp;
  }
  a.targets = targets;
  a.target_bytes = target_bytes;
  a.vocab = vocab;
  a.part_max = (float*)(ws + p.pmax);
  a.part_sum = (float*)(ws + p.psum);
  a.target_logit = (float*)(ws + p.tlogit);
  launch<kStats>(a, p.small, dtype, 1, s);
  if (int rc = launched(who)) return rc;
  join_stats_kernel<<<dim3((uint32_t)((tokens + 15) / 16)), dim3(256), 0, s>>>(
      a.part_max, a.part_sum, a.target_logit, targets, target_bytes, tokens, vocab,
      (int32_t)p.parts, loss, lse);
  return launched(who);
}

extern "C" int zs_xent_backward(const void* hidden, int64_t hidden_stride, const void* weight,
                                int64_t weight_stride, const void* targets, const float* lse,
                                const float* grad_loss, void* grad_hidden,
                                int64_t grad_hidden_stride, void* grad_weight,
                                int64_t grad_weight_stride, int64_t tokens, int64_t vocab,
                                int64_t width, int32_t dtype, int32_t target_bytes,
                                void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "zs_xent_backward";
  if (int rc = check(who, hidden, hidden_stride, weight, weight_stride, targets, tokens, vocab,
                     width, dtype, target_bytes))
    return rc;
  if ((grad_hidden && grad_hidden_stride < width) || (grad_weight && grad_weight_stride < width))
    return fail(who, "a row stride is below width");
  if (tokens > kMaxStride - 64) return fail(who, "too many tokens for one call");
  if (tokens && (!lse || !grad_loss)) return fail(who, "NULL buffer");
  if (!al(lse, 4) || !al(grad_loss, 4) || !al(grad_hidden, 2) || !al(grad_weight, 2))
    return fail(who, "a buffer is not aligned to its elements");
  const Plan p = plan(hidden, hidden_stride, weight, weight_stride, tokens, vocab, width, true);
  if (!workspace || !al(workspace, 256)) return fail(who, "the workspace is NULL or not 256-byte aligned");
  if (workspace_bytes < p.total) return fail(who, "the workspace is too small");
  GemmArgs lg{}, gw{}, gh{};
  const int64_t per_row = (p.wp / 4 + 255) / 256;
  if (!shape(&lg, p.small, p.piece, std::max<int64_t>(tokens, 1), p.wp, 1) ||
      !shape(&gw, false, width, p.piece, std::max<int64_t>(tokens, 8), 1) ||
      !shape(&gh, p.small, width, std::max<int64_t>(tokens, 1), p.piece, p.splits) ||
      per_row * tokens > 0xffffff)
    return fail(who, "too many rows for one call");
  if (!grad_hidden && !grad_weight) return ZS_OK;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* ws = (uint8_t*)workspace;
  const uint16_t *h = (const uint16_t*)hidden, *w = (const uint16_t*)weight;
  int64_t ldh = hidden_stride, ldw = weight_stride;
  float* gmax = (float*)(ws + p.gmax);
  uint16_t *ht = (uint16_t*)(ws + p.ht), *wt = (uint16_t*)(ws + p.wt), *g = (uint16_t*)(ws + p.g),
           *gt = (uint16_t*)(ws + p.gt);
  float* acc = (float*)(ws + p.acc);
  if (p.copy_w) {
    copy_rows(weight, weight_stride, vocab, width, ws + p.w, p.wp, s);
    w = (const uint16_t*)(ws + p.w);
    ldw = p.wp;
  }
  if (p.copy_h) {
    copy_rows(hidden, hidden_stride, tokens, width, ws + p.h, p.wp, s);
    h = (const uint16_t*)(ws + p.h);
    ldh = p.wp;
  }
  gmax_kernel<<<dim3(1), dim3(1024), 0, s>>>(grad_loss, targets, target_bytes, tokens, vocab, gmax);
  const uint32_t wt_cols = (uint32_t)((width + 63) / 64);
  if (grad_weight)
    transpose_kernel<<<dim3((uint32_t)(p.tp / 64), wt_cols), dim3(256), 0, s>>>(
        h, ldh, tokens, width, ht, p.tp, p.tp, targets, target_bytes, vocab);
  if (int rc = launched(who)) return rc;
  for (int64_t v0 = 0; v0 < vocab; v0 += p.piece) {
    const int64_t rows = std::min(p.piece, vocab - v0), cols = up(rows, 8);
    if (tokens) {
      GemmArgs a{};
      shape(&a, p.small, rows, tokens, p.wp, 1);
      a.a = w + v0 * ldw;
      a.lda = ldw;
      a.b = h;
      a.ldb = ldh;
      a.targets = targets;
      a.target_bytes = target_bytes;
      a.vocab = vocab;
      a.v0 = v0;
      a.lse = lse;
      a.gloss = grad_loss;
      a.gmax = gmax;
      a.g = g;
      a.ldg = cols;
      a.gt = grad_weight ? gt : nullptr;
      a.ldgt = p.tp;
      a.n_pad = p.tp;
      launch<kGrad>(a, p.small, dtype, 1, s);
    }
    if (grad_weight) {
      GemmArgs a{};
      shape(&a, false, width, rows, tokens ? p.tp : 0, 1);
      a.a = ht;
      a.lda = p.tp;
      a.b = gt;
      a.ldb = p.tp;
      a.gmax = gmax;
      a.c = (uint16_t*)grad_weight + v0 * grad_weight_stride;
      a.ldc = grad_weight_stride;
      a.c_wide = wide(grad_weight, grad_weight_stride, dtype);
      launch<kStore>(a, false, dtype, 1, s);
    }
    if (grad_hidden && tokens) {
      transpose_kernel<<<dim3((uint32_t)((cols + 63) / 64), wt_cols), dim3(256), 0, s>>>(
          w + v0 * ldw, ldw, rows, width, wt, cols, cols, nullptr, 8, vocab);
      GemmArgs a{};
      shape(&a, p.small, width, tokens, cols, p.splits);
      a.a = wt;
      a.lda = cols;
      a.b = g;
      a.ldb = cols;
      a.acc = acc;
      a.ldc = p.wp;
      a.acc_split = tokens * p.wp;
      a.add = v0 > 0;
      launch<kAccum>(a, p.small, dtype, p.splits, s);
    }
    if (int rc = launched(who)) return rc;
  }
  if (grad_hidden && tokens) {
    auto go = [&](auto DT) {
      constexpr int D = decltype(DT)::value;
      finish_kernel<D><<<dim3((uint32_t)(per_row * tokens)), dim3(256), 0, s>>>(
          acc, p.wp, tokens * p.wp, p.splits, gmax, (elem_t<D>*)grad_hidden, grad_hidden_stride,
          tokens, width, (int32_t)per_row);
    };
    if (dtype == ZS_BF16)
      go(std::integral_constant<int, ZS_BF16>());
    else
      go(std::integral_constant<int, ZS_F16>());
  }
  return launched(who);
}
