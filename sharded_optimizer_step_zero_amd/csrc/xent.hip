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
// tile); a second kernel joins them.  Backward: pieces of the vocabulary; for each,
// the product again, its tiles ending in G, and the two products that use it.
// 8 * tokens * vocab * width operations in all, on the matrix cores: bound by
// their rate where there are tokens enough, by reading W where there are few.
//
// All three products are one kernel, C[n][m] = sum_k A[m][k] B[n][k], on 16x16x32
// matrix instructions (16-bit in, fp32 sums).  An operand lies in memory with k
// adjacent (H and W for the logits, G for dH) or with its rows adjacent (W for dH,
// H and G for dW), so nothing is transposed on the way: the second kind goes
// through the LDS reads that transpose.
//
// 256 x 256 tiles, four waves of 128 x 128 each: a wave reads 16 operand
// fragments of LDS for 64 matrix instructions, which leaves the LDS less busy
// than the matrix cores (eight waves of 128 x 64, with W, H and G transposed on the
// way, took 8.3 ms where this takes 6.7).  Tiles of 64 k, two in LDS, come from
// global memory straight into it.  A step multiplies a tile's first 32 k while it reads
// the fragments of the second, then the second while it reads the next tile's
// first, so no multiplication waits for LDS; between the two halves is the step's
// one barrier, where the next tile's loads, started a step before, have landed and
// this tile's buffer is free for the loads of the one after.  Few tokens, or few
// tiles, take 128 x 64 tiles of four waves and three buffers instead.
//
// A row with k adjacent takes 128 bytes of LDS, a cache line of memory (with 64 bytes a
// row and four buffers: 7.06 against 6.85 ms); its 16-byte chunk c sits at c ^ (row
// & 7), so that 8 neighbouring rows' chunks lie on different banks.  Where rows are
// adjacent, chunk c of k's line sits at c ^ 2 * ((k & 3) | ((k >> 3) & 1) << 2): the
// lines that one transposing read meets differ (no bank conflicts counted in the
// loops).  Rows past the edge and k past the end read as zeros by the buffer loads'
// bounds check.
//
// Measured, 8192 tokens x 4096 x 32000 bf16: loss 1.68 ms (1280 TFLOP/s), loss and
// gradients 6.74 ms (1270 TFLOP/s of the 8 tokens vocab width operations done; the
// library's bare product 1370 to 1430).  The clock gives way under the load: on
// zeros the same loop runs at 1650.  32x32x16 instructions are faster on zeros (1745) and
// slower on data (1190).  64 x 2048 x 50304: 46 us of reading W at 4.5 TB/s, and 5 joining.
#include <algorithm>

#include "ops.h"
#include "xent_plan.h"

namespace zs {
namespace ops {
namespace {

typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
#define ZS_LDS __attribute__((address_space(3)))

constexpr int kRsrcWord3 = 0x00020000;  // raw 32-bit buffer, gfx9 family
constexpr int BK = 64;  // k elements of one step

// what a tile ends in
constexpr int kStats = 0;   // maximum, sum of exponentials and target logit
constexpr int kGrad = 1;    // G
constexpr int kStore = 2;   // C, rounded
constexpr int kAccum = 3;   // C in fp32, stored or added
// how an operand lies
constexpr int kByK = 0;     // [row][k]
constexpr int kByRow = 1;   // [k][row]

struct GemmArgs {
  const uint16_t *a, *b;
  int64_t lda, ldb;      // strides, multiples of 8; a line's last chunk is whole in memory
  int64_t m, n, k;       // rows of A and of B, and k
  int32_t tiles_m, tiles_n;
  int64_t k_per_split;   // a multiple of BK
  // kStats, kGrad
  const void* targets;
  int32_t target_bytes;
  int64_t vocab, v0;     // A's first row is vocabulary entry v0
  float *part_max, *part_sum, *target_logit;
  const float *lse, *gloss, *gmax;
  uint16_t* g;           // G [n][ldg], whole rows
  int64_t ldg;
  // kStore, kAccum
  uint16_t* c;
  float* acc;
  int64_t ldc, acc_split;
  int32_t add, c_wide;
};

// c += a b on the matrix cores, c held in the accumulation registers: left to
// itself the compiler spreads 256 sums over both register files and moves them
// to and fro.  It does not know how long the result takes, so settle() has to
// come before anything else touches the sums: at the end of a loop's body, which
// itself has matrix instructions only.
template <int DT>
__device__ __forceinline__ void mfma(f32x4& c, s16x8 a, s16x8 b) {
  if constexpr (DT == ZS_BF16)
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  else
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
// The last matrix instruction's result is written (18 wait states after its issue).
__device__ __forceinline__ void settle() { asm volatile("s_nop 15\n\ts_nop 3" ::: "memory"); }
template <int DT>
__device__ __forceinline__ uint16_t round16(float x) {
  return __builtin_bit_cast(uint16_t, (elem_t<DT>)x);
}

template <int DT>
__device__ __forceinline__ u32x2 pack16(f32x4 x) {
  typedef elem_t<DT> v4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(u32x2, __builtin_convertvector(x, v4));
}
constexpr float kLog2E = 1.44269504f;
// G's largest magnitude.  Most of a softmax lies far below its targets, and fp16 has digits
// down to 2^-14 only, but fifteen binades above 1 that nothing else would use: improbable
// entries keep the digits they would lose, at no cost, as the factor comes back together
// with grad_loss.  (A power of two: exact.  At 2^15 an error in p of any size below 1 still fits.)
template <int DT>
constexpr float kTopG = DT == ZS_F16 ? 0x1p15f : 1.0f;
// e^(x - y).  The difference comes first: where x is y the result is 1, so that a sum whose
// maximum stays is joined unchanged however often.  (With y log2 e rounded beforehand, each
// join multiplied by 1 + |y| 2^-24 or so: a token sure of its target was off by 20 units in
// its lse, and p - 1 there could be positive.)
__device__ __forceinline__ float exp_of(float x, float y) {
  return __builtin_amdgcn_exp2f((x - y) * kLog2E);
}
// Many e^(x - y) of one y, in one fused step each, x log2 e - power, and what y log2 e lost
// when it was rounded as a factor of them all.  (The difference first costs an instruction
// an entry: 0.5% of the loss and gradients at 1003 x 1000 x 32003.)
struct Under {
  float power, factor;
  __device__ __forceinline__ explicit Under(float y) {
    power = y * kLog2E;
    factor = __builtin_amdgcn_exp2f(-__builtin_fmaf(y, kLog2E, -power));
  }
  __device__ __forceinline__ float operator()(float x) const {  // e^(x - y) / factor
    return __builtin_amdgcn_exp2f(__builtin_fmaf(x, kLog2E, -power));
  }
};
// A maximum to take differences from, also where nothing has come yet: e^-infinity is 0.
__device__ __forceinline__ float base_of(float top) {
  return top == -__builtin_inff() ? 0.0f : top;
}

__device__ __forceinline__ int64_t target_of(const GemmArgs& g, int64_t t) {
  return g.target_bytes == 8 ? ((const int64_t*)g.targets)[t] : ((const int32_t*)g.targets)[t];
}

// The tile of a workgroup, and its part of k.  Workgroups go round the 8 dies: each die
// takes a contiguous part of the tiles of all splits, split by split, which run down
// a band of 8 tiles of B, so that the tiles at work on a die share their rows of A
// and B in its L2.
__device__ __forceinline__ void tile_of(const GemmArgs& g, int32_t* tm, int32_t* tn,
                                        int32_t* split) {
  const uint32_t tiles = (uint32_t)g.tiles_m * (uint32_t)g.tiles_n, total = gridDim.x;
  const uint32_t die = blockIdx.x & 7, per = total >> 3, extra = total & 7;
  const uint32_t all = die * per + (die < extra ? die : extra) + (blockIdx.x >> 3);
  *split = (int32_t)(all / tiles);
  const uint32_t id = all - (uint32_t)*split * tiles;
  const uint32_t band = id / ((uint32_t)g.tiles_m * 8);
  const uint32_t in = id - band * (uint32_t)g.tiles_m * 8;
  const uint32_t wide = (uint32_t)g.tiles_n - band * 8 < 8 ? (uint32_t)g.tiles_n - band * 8 : 8;
  *tm = (int32_t)(in / wide);
  *tn = (int32_t)(band * 8 + in % wide);
}

// One operand's way from memory through LDS into a wave's fragments: R rows a
// tile, F fragments of 16 rows a wave, `threads` threads.
template <int LAYOUT, int R, int F, int THREADS>
struct Operand {
  static constexpr int kBytes = R * BK * 2;
  static constexpr int kLoads = kBytes / (THREADS * 16);  // of a thread, for a tile
  static_assert(kBytes % (THREADS * 16) == 0, "whole loads");
  static constexpr int kLine = LAYOUT == kByK ? BK * 2 : R * 2;  // bytes of a line in LDS
  static constexpr int kChunks = kLine / 16;
  static constexpr int kLinesPerLoad = THREADS / kChunks;
  static_assert(LAYOUT == kByK || kLinesPerLoad % 4 == 0, "k & 3 does not depend on the load");

  const uint8_t* base;   // the tile's first element at the split's first k
  int64_t ld;            // bytes
  int32_t rows, k_len;   // that exist
  uint32_t off[kLoads];  // a thread's place in each load
  int32_t chunk_k;       // kByK: the first k of the thread's chunk

  __device__ __forceinline__ static int swizzle(int line) {
    if (LAYOUT == kByK) return line & 7;
    return ((line & 3) | ((line >> 3) & 1) << 2) * 2 & (kChunks - 1);
  }
  __device__ __forceinline__ Operand(const uint16_t* p, int64_t stride, int64_t row0,
                                     int64_t n_rows, int64_t k0, int32_t k, int tid) {
    ld = stride * 2;
    base = (const uint8_t*)(LAYOUT == kByK ? p + row0 * stride + k0 : p + k0 * stride + row0);
    rows = (int32_t)(n_rows - row0 < R ? n_rows - row0 : R);
    k_len = k;
    const int line = tid / kChunks, at = tid % kChunks;
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      const int l = line + i * kLinesPerLoad;
      off[i] = (uint32_t)(l * ld + (at ^ swizzle(l)) * 16);
    }
    // kLinesPerLoad is a multiple of 8 here: the chunk is the same in every load
    chunk_k = (at ^ swizzle(line)) * 8;
  }
  // Buffer descriptor of step `step`'s tile: what lies past it reads as zeros.
  __device__ __forceinline__ u32x4 descriptor(int step) const {
    const int32_t left = k_len - step * BK;
    const uint8_t* p = base + (LAYOUT == kByK ? (int64_t)step * BK * 2 : step * BK * ld);
    const int32_t lines = left < BK ? left : BK;
    // up to the end of the last line's last chunk, which the stride covers
    const int64_t bytes = LAYOUT == kByK ? (rows - 1) * ld + ((left + 7) & ~7) * 2
                                         : (int64_t)(lines - 1) * ld + ((rows + 7) & ~7) * 2;
    const uint64_t q = (uint64_t)p;
    const uint32_t end = left > 0 ? (uint32_t)bytes : 0u;
    // the same in every lane, which the compiler does not always see
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)q),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)(q >> 32)),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)end), (uint32_t)kRsrcWord3};
  }
  // Before the loads of step `step`: k past the end would be the next row's, so in
  // the last tile a thread whose chunk is past it reads out of bounds.
  __device__ __forceinline__ void limit(int step) {
    const int32_t left = k_len - step * BK;
    if (LAYOUT == kByK && left < BK) {
#pragma unroll
      for (int i = 0; i < kLoads; i++) off[i] = chunk_k < left ? off[i] : 0xfffffff0u;
    }
  }
  // The same for one load, where the tiles do not come in order.
  __device__ __forceinline__ uint32_t limited(int step, int i) const {
    return LAYOUT == kByK && chunk_k >= k_len - step * BK ? 0xfffffff0u : off[i];
  }
  // Load i of the tile, into LDS at `lds` (the wave's part of the load).  The compiler does not
  // see a load here: a descriptor's scalar that a vector instruction wrote would have to be
  // five wait states old.  Descriptors come from the scalar side; test_ops_assembly_hazards.py
  // looks whether any build brings one closer (a wait here costs the loop 0.7%).
  __device__ __forceinline__ void load(u32x4 d, int i, uint32_t lds) const {
    load(d, off[i], i, lds);
  }
  __device__ __forceinline__ void load(u32x4 d, uint32_t from, int i, uint32_t lds) const {
    // m0 is the compiler's own, which it warns of: it has to know that its value is gone
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
    asm volatile(
        "s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(
            lds + i * THREADS * 16),
        "v"(from), "s"(d)
        : "memory", "m0");
#pragma clang diagnostic pop
  }
  // Fragment f of the tile's half `half`, for the wave whose first row is `row0`: 16
  // rows and 32 k; a lane has 8 k of one row.
  __device__ __forceinline__ static s16x8 fragment(const uint8_t* tile, int half, int f, int row0,
                                                   int lane) {
    if constexpr (LAYOUT == kByK) {
      const int row = row0 + (lane & 15), chunk = (half * 4 + (lane >> 4)) ^ swizzle(row);
      // 16 rows on, the swizzle is the same
      return *(const s16x8*)(tile + row * kLine + chunk * 16 + f * 16 * kLine);
    } else {
      // 16 lanes read 4 lines of k, 16 rows each, and get a row's 4 k each
      const int k = half * 32 + (lane >> 4) * 8 + ((lane & 15) >> 2);
      const int row = row0 + f * 16 + (lane & 3) * 4;
      const int chunk = (row >> 3) ^ swizzle(k);
      const uint8_t* p = tile + k * kLine + chunk * 16 + (row & 4) * 2;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZS_LDS s16x4*)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZS_LDS s16x4*)(p + 4 * kLine));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

template <int DT, int LA, int LB, int BM, int BN, int WM, int WN, int kBuffers, int EPI>
__device__ __forceinline__ void gemm(const GemmArgs& g) {
  constexpr int kThreads = WM * WN * 64;
  constexpr bool kTurned = BN == 64;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  using OpA = Operand<LA, BM, FM, kThreads>;
  using OpB = Operand<LB, BN, FN, kThreads>;
  constexpr int kTile = OpA::kBytes + OpB::kBytes;
  constexpr int kLoads = OpA::kLoads + OpB::kLoads;
  static_assert(kBuffers * kTile >= BM * BN * 2 && kBuffers * kTile >= WM * BN * 8,
                "the epilogue's tile fits");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kBuffers * kTile];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  int32_t tm, tn, split;
  tile_of(g, &tm, &tn, &split);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int64_t k_begin = split * g.k_per_split;
  const int64_t k_end = k_begin + g.k_per_split < g.k ? k_begin + g.k_per_split : g.k;
  const int32_t k_len = k_end > k_begin ? (int32_t)(k_end - k_begin) : 0;
  const int steps = (k_len + BK - 1) / BK;

  OpA a(g.a, g.lda, m0, g.m, k_begin, k_len, tid);
  OpB b(g.b, g.ldb, n0, g.n, k_begin, k_len, tid);
  const uint32_t lds_at = (uint32_t)(uintptr_t)(ZS_LDS uint8_t*)lds + wave * 1024;

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int j = 0; j < FN; j++) acc[i][j] = f32x4{};

  const int ra = wm * (BM / WM), rb = wn * (BN / WN);

  // the loads of a step's tile, past the last step too (zeros), so that their
  // number is always the same
  auto load = [&](int buffer, int step, int i, u32x4 da, u32x4 db) {
    const uint32_t to = lds_at + buffer * kTile;
    const bool of_a = i < OpA::kLoads;
    if (!of_a) i -= OpA::kLoads;
    if (kTurned && of_a)
      a.load(da, a.limited(step, i), i, to);
    else if (kTurned)
      b.load(db, b.limited(step, i), i, to + OpA::kBytes);
    else if (of_a)
      a.load(da, i, to);
    else
      b.load(db, i, to + OpA::kBytes);
  };
  // The tile of step s.  With few tokens the products are bound by memory, and rows at a
  // multiple of 4 KB would have all workgroups read one column, which few of the
  // memory's channels hold: there every workgroup begins at a step of its own.
  const int turn = kTurned && steps > 0 ? (int)((uint32_t)(tm + split) * 5u % (uint32_t)steps) : 0;
  auto turned = [&](int s) {
    if (!kTurned || s >= steps) return s;
    const int at = s + turn;
    return at < steps ? at : at - steps;
  };
  // Multiplies fragments fa, fb while half `half` of the tile at `tile` is read into
  // ga, gb, and (loads) starts the loads of step `ahead` into `buffer`.  Reads, in the
  // order in which the next half needs them, and loads are dealt out between
  // pairs of matrix instructions, which take longer than issuing them; the last
  // eighth has none, so that the last reads have arrived.
  auto multiply = [&](s16x8 (&fa)[FM], s16x8 (&fb)[FN], s16x8 (&ga)[FM], s16x8 (&gb)[FN],
                      const uint8_t* tile, int half, bool loads, int buffer, int ahead) {
    u32x4 da = {}, db = {};
    if (loads) {
      ahead = turned(ahead);
      if (!kTurned) {
        a.limit(ahead);
        b.limit(ahead);
      }
      da = a.descriptor(ahead);
      db = b.descriptor(ahead);
    }
    constexpr int kPairs = FM * FN / 2, kSpan = kPairs * 7 / 8, kReads = FM + FN;
    const int n_loads = loads ? kLoads : 0;
#pragma unroll
    for (int x = 0; x < kPairs; x++) {
#pragma unroll
      for (int e = (x * kReads + kSpan - 1) / kSpan;
           e < ((x + 1) * kReads + kSpan - 1) / kSpan && e < kReads; e++) {
        if (e == 0)
          ga[0] = OpA::fragment(tile, half, 0, ra, lane);
        else if (e <= FN)
          gb[e - 1] = OpB::fragment(tile + OpA::kBytes, half, e - 1, rb, lane);
        else
          ga[e - FN] = OpA::fragment(tile, half, e - FN, ra, lane);
      }
#pragma unroll
      for (int e = (x * n_loads + kSpan - 1) / kSpan;
           e < ((x + 1) * n_loads + kSpan - 1) / kSpan && e < n_loads; e++)
        load(buffer, ahead, e, da, db);
#pragma unroll
      for (int y = 2 * x; y < 2 * x + 2; y++) {
        // to and fro, so that a turn keeps both a row's and a column's operand
        const int i = y / FN, j = i & 1 ? FN - 1 - y % FN : y % FN;
        mfma<DT>(acc[i][j], fa[i], fb[j]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  if (steps > 0) {
#pragma unroll
    for (int t = 0; t < kBuffers; t++) {
      const int from = turned(t);
      if (!kTurned) {
        a.limit(from);
        b.limit(from);
      }
      const u32x4 da = a.descriptor(from), db = b.descriptor(from);
#pragma unroll
      for (int l = 0; l < kLoads; l++) load(t, from, l, da, db);
    }
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((kBuffers - 1) * kLoads) : "memory");
    s16x8 fa[FM], fb[FN], ga[FM], gb[FN];
#pragma unroll
    for (int i = 0; i < FM; i++) fa[i] = OpA::fragment(lds, 0, i, ra, lane);
#pragma unroll
    for (int j = 0; j < FN; j++) fb[j] = OpB::fragment(lds + OpA::kBytes, 0, j, rb, lane);
    int buffer = 0;
    for (int s = 0; s < steps; s++) {
      const int next = buffer + 1 < kBuffers ? buffer + 1 : 0;
      multiply(fa, fb, ga, gb, lds + buffer * kTile, 1, false, 0, 0);
      // tile s + 1 has landed for every wave, and every wave has read tile s
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((kBuffers - 2) * kLoads)
                   : "memory");
      multiply(ga, gb, fa, fb, lds + next * kTile, 0, true, buffer, s + kBuffers);
      settle();
      buffer = next;
    }
  }
  // no load is on its way into LDS any more, and no wave reads it
  asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");

  // acc[i][j][r] is C at row m0 + wm*(BM/WM) + i*16 + (lane>>4)*4 + r of A and row
  // n0 + wn*(BN/WN) + j*16 + (lane&15) of B
  const int em = wm * (BM / WM) + (lane >> 4) * 4, en = wn * (BN / WN) + (lane & 15);

  // entries past the vocabulary (the last tile's) take no part
  if (EPI == kStats && m0 + BM > g.vocab) {
    const int32_t left = (int32_t)(g.vocab - m0) - em;
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
      for (int r = 0; r < 4; r++)
        if (i * 16 + r >= left) {
#pragma unroll
          for (int j = 0; j < FN; j++) acc[i][j][r] = -__builtin_inff();
        }
  }
  // A token's target as i * 16 + r, where this lane has it; -1 elsewhere.
  auto mine = [&](int64_t target) {
    const int64_t at = target - (g.v0 + m0 + em);
    return target < g.vocab && at >= 0 && at < FM * 16 && !(at & 12) ? (int)at : -1;
  };

  if constexpr (EPI == kStats) {
    f32x2* stats = (f32x2*)lds;
#pragma unroll
    for (int j = 0; j < FN; j++) {
      const int64_t t = n0 + en + j * 16;
      const int at = t < g.n ? mine(target_of(g, t)) : -1;
      if (at >= 0) {
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
          for (int r = 0; r < 4; r++)
            if (at == i * 16 + r) g.target_logit[t] = acc[i][j][r];
      }
      float top = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < FM; i++)
#pragma unroll
        for (int r = 0; r < 4; r++) top = __builtin_fmaxf(top, acc[i][j][r]);
      top = __builtin_fmaxf(top, __shfl_xor(top, 16, 64));
      top = __builtin_fmaxf(top, __shfl_xor(top, 32, 64));
      const Under under(base_of(top));
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < FM; i++)
#pragma unroll
        for (int r = 0; r < 4; r++) sum += under(acc[i][j][r]);
      sum += __shfl_xor(sum, 16, 64);
      sum += __shfl_xor(sum, 32, 64);
      sum *= under.factor;
      // the maximum's own exponential is 1: what is below is rounding, and a loss is not negative
      if (sum < 1.0f && top > -__builtin_inff()) sum = 1.0f;
      if (lane < 16) stats[wm * BN + en + j * 16] = f32x2{top, sum};
    }
    __syncthreads();
    for (int i = tid; i < BN; i += kThreads) {  // the waves of one token, in order
      float top = stats[i][0];
#pragma unroll
      for (int w = 1; w < WM; w++) top = __builtin_fmaxf(top, stats[w * BN + i][0]);
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < WM; w++)
        sum += stats[w * BN + i][1] * exp_of(stats[w * BN + i][0], base_of(top));
      if (n0 + i < g.n) {
        g.part_max[tm * g.n + n0 + i] = top;
        g.part_sum[tm * g.n + n0 + i] = sum;
      }
    }
  } else if constexpr (EPI == kAccum) {
    float* out = g.acc + split * g.acc_split;
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
    const float factor = *g.gmax;
    auto to = [&](int row, int m) {
      return lds + row * (BM * 2) + ((m >> 3) ^ (row & (BM / 8 - 1))) * 16 + (m & 7) * 2;
    };
#pragma unroll
    for (int j = 0; j < FN; j++) {
      const int row = en + j * 16;
      const int64_t t = n0 + row;
      float lse = 0.0f, scale = factor;
      bool counts = true;
      int at = -1;
      if (EPI == kGrad) {
        const int64_t target = t < g.n ? target_of(g, t) : -1;
        counts = target >= 0 && target < g.vocab;
        if (counts) {
          lse = g.lse[t];
          scale = g.gloss[t] / factor * kTopG<DT>;
          at = mine(target);
        }
      }
      const Under under(lse);
      const float each = EPI == kGrad ? scale * under.factor : scale;
#pragma unroll
      for (int i = 0; i < FM; i++) {
        f32x4 x;
#pragma unroll
        for (int r = 0; r < 4; r++)
          x[r] = (EPI == kGrad ? under(acc[i][j][r]) : acc[i][j][r] / kTopG<DT>) * each;
        u32x2 w = pack16<DT>(x);
        if (EPI == kGrad && !counts) w = u32x2{0, 0};
        *(u32x2*)to(row, em + i * 16) = w;
      }
      if (EPI == kGrad && at >= 0) {  // this lane wrote that place
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
          for (int r = 0; r < 4; r++)
            if (at == i * 16 + r)
              *(uint16_t*)to(row, em + at) =
                  round16<DT>((exp_of(acc[i][j][r], lse) - 1.0f) * scale);
      }
    }
    if (EPI == kGrad && g.v0 + m0 + BM > g.vocab) {  // zeros past the vocabulary
      __syncthreads();
      const int first = (int)(g.vocab - g.v0 - m0);
      for (int x = tid; x < BM * BN; x += kThreads)
        if (x % BM >= first) *(uint16_t*)to(x / BM, x % BM) = 0;
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
  }
}

template <int DT, int LA, int LB, int BM, int BN, int WM, int WN, int kBuffers, int EPI>
__global__ __launch_bounds__(WM* WN * 64, 1) void gemm_kernel(GemmArgs g) {
  gemm<DT, LA, LB, BM, BN, WM, WN, kBuffers, EPI>(g);
}

// Joins a token's partial maxima and sums: 64 threads a token, each over every
// 64th part in order, then the threads in pairs.
__global__ __launch_bounds__(1024) void join_stats_kernel(
    const float* __restrict__ part_max, const float* __restrict__ part_sum,
    const float* __restrict__ target_logit, const void* __restrict__ targets,
    int32_t target_bytes, int64_t tokens, int64_t vocab, int32_t parts, float* __restrict__ loss,
    float* __restrict__ lse) {
  __shared__ float tops[16][16], sums[16][16];
  const int tt = threadIdx.x & 15, s = threadIdx.x >> 4;
  const int64_t t = (int64_t)blockIdx.x * 16 + tt;
  // a part of nothing but -infinity, and no part at all, has the sum 0
  auto join = [](float& top, float& sum, float m, float x) {
    const float next = __builtin_fmaxf(top, m);
    sum = sum * exp_of(top, base_of(next)) + x * exp_of(m, base_of(next));
    top = next;
  };
  float top = -__builtin_inff(), sum = 0.0f;
  if (t < tokens) {
#pragma unroll 8
    for (int p = s; p < parts; p += 64)
      join(top, sum, part_max[p * tokens + t], part_sum[p * tokens + t]);
  }
  for (int d = 16; d < 64; d <<= 1)  // the wave's four threads of the token
    join(top, sum, __shfl_xor(top, d, 64), __shfl_xor(sum, d, 64));
  if ((threadIdx.x & 63) < 16) {
    tops[threadIdx.x >> 6][tt] = top;
    sums[threadIdx.x >> 6][tt] = sum;
  }
  __syncthreads();
  if (threadIdx.x >= 64) return;
  top = -__builtin_inff();
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; i++) join(top, sum, tops[s * 4 + i][tt], sums[s * 4 + i][tt]);
  for (int d = 16; d < 64; d <<= 1) join(top, sum, __shfl_xor(top, d, 64), __shfl_xor(sum, d, 64));
  if (s != 0 || t >= tokens) return;
  const float l = sum == 0.0f ? -__builtin_inff() : __builtin_logf(sum);
  const int64_t target =
      target_bytes == 8 ? ((const int64_t*)targets)[t] : ((const int32_t*)targets)[t];
  lse[t] = l + top;
  // not lse - logit: a small loss would be what lse's rounding leaves
  loss[t] = target >= 0 && target < vocab ? l + (top - target_logit[t]) : 0.0f;
}

// Rows copied to a stride that is a multiple of 8 elements, zeros past the width.
// With targets: zeros for the rows of tokens that do not count, whatever they hold,
// and one more workgroup finds the largest finite |grad_loss| of those that do (1
// where that is 0).
__global__ __launch_bounds__(256) void copy_rows_kernel(
    const uint16_t* __restrict__ in, int64_t in_stride, int64_t rows, int64_t width,
    uint16_t* __restrict__ out, int64_t out_stride, const void* __restrict__ targets,
    int32_t target_bytes, int64_t vocab, const float* __restrict__ gloss,
    float* __restrict__ gmax) {
  auto counts = [&](int64_t r) {
    const int64_t t =
        target_bytes == 8 ? ((const int64_t*)targets)[r] : ((const int32_t*)targets)[r];
    return t >= 0 && t < vocab;
  };
  if (gmax && blockIdx.x == 0) {
    __shared__ float slots[4];
    float top = 0.0f;
#pragma unroll 4
    for (int64_t t = threadIdx.x; t < rows; t += 256) {
      const float x = __builtin_fabsf(gloss[t]);
      if (counts(t) && x < __builtin_inff()) top = __builtin_fmaxf(top, x);
    }
    for (int d = 1; d < 64; d <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d, 64));
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < 4; i++) top = __builtin_fmaxf(top, slots[i]);
      *gmax = top > 0.0f ? top : 1.0f;
    }
    return;
  }
  const int64_t skip = gmax ? 1 : 0;
  for (int64_t r = blockIdx.x - skip; r < rows; r += gridDim.x - skip) {
    const bool kept = !targets || counts(r);
    for (int64_t c = threadIdx.x * 8; c < out_stride; c += 256 * 8) {
      const Chunk<ZS_BF16> x =
          load_chunk<ZS_BF16>((const __bf16*)in + r * in_stride + c, kept ? width - c : 0);
      *(u32x4*)(out + r * out_stride + c) = x.w[0];
    }
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
  s = s / kTopG<DT> * *gmax;
  for (int i = 0; i < 4; i++)
    if (c + i < width) out[row * out_stride + c + i] = (elem_t<DT>)s[i];
}

// ---------------------------------------------------------------- host side

constexpr int64_t kMaxWidth = 65536, kMaxStride = 1 << 21, kMaxRows = 0x7fffffff - 512;
using xent::Plan;
using xent::plan;
using xent::up;

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

template <int EPI, int LA, int LB>
void launch(const GemmArgs& a, bool small, int dtype, int splits, hipStream_t s) {
  const dim3 grid((uint32_t)a.tiles_m * (uint32_t)a.tiles_n * (uint32_t)splits);
  auto go = [&](auto DT) {
    constexpr int D = decltype(DT)::value;
    if (small)
      gemm_kernel<D, LA, LB, 128, 64, 4, 1, 3, EPI><<<grid, dim3(256), 0, s>>>(a);
    else
      gemm_kernel<D, LA, LB, 256, 256, 2, 2, 2, EPI><<<grid, dim3(256), 0, s>>>(a);
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
  return tm * tn * splits * 512 <= 0xffffffffll;
}

void copy_rows(const void* in, int64_t stride, int64_t rows, int64_t width, void* out,
               int64_t wp, hipStream_t s) {
  if (rows)
    copy_rows_kernel<<<dim3((uint32_t)std::min<int64_t>(rows, 8192)), dim3(256), 0, s>>>(
        (const uint16_t*)in, stride, rows, width, (uint16_t*)out, wp, nullptr, 8, 0, nullptr,
        nullptr);
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
  const int64_t join_blocks = (tokens + 15) / 16;
  if (!shape(&a, p.small, vocab, tokens, p.wp, 1) || join_blocks * 1024 > 0xffffffffll)
    return fail(who, "too many rows for one call");
  hipStream_t s = (hipStream_t)stream;
  uint8_t* ws = (uint8_t*)workspace;
  a.a = (const uint16_t*)weight;
  a.lda = weight_stride;
  a.b = (const uint16_t*)hidden;
  a.ldb = hidden_stride;
  if (p.copy_w) {
    copy_rows(weight, weight_stride, vocab, width, ws + p.w, p.cs, s);
    a.a = (const uint16_t*)(ws + p.w);
    a.lda = p.cs;
  }
  if (p.copy_h) {
    copy_rows(hidden, hidden_stride, tokens, width, ws + p.h, p.cs, s);
    a.b = (const uint16_t*)(ws + p.h);
    a.ldb = p.cs;
  }
  a.targets = targets;
  a.target_bytes = target_bytes;
  a.vocab = vocab;
  a.part_max = (float*)(ws + p.pmax);
  a.part_sum = (float*)(ws + p.psum);
  a.target_logit = (float*)(ws + p.tlogit);
  launch<kStats, kByK, kByK>(a, p.small, dtype, 1, s);
  if (int rc = launched(who)) return rc;
  join_stats_kernel<<<dim3((uint32_t)join_blocks), dim3(1024), 0, s>>>(
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
      !shape(&gw, p.small_w, width, p.piece, std::max<int64_t>(tokens, 8), 1) ||
      !shape(&gh, p.small_h, width, std::max<int64_t>(tokens, 1), p.piece, p.splits) ||
      per_row * tokens > 0xffffff)
    return fail(who, "too many rows for one call");
  if (!grad_hidden && !grad_weight) return ZS_OK;
  hipStream_t s = (hipStream_t)stream;
  uint8_t* ws = (uint8_t*)workspace;
  const uint16_t *h = (const uint16_t*)(ws + p.h), *w = (const uint16_t*)weight;
  int64_t ldw = weight_stride;
  float* gmax = (float*)(ws + p.gmax);
  uint16_t* g = (uint16_t*)(ws + p.g);
  float* acc = (float*)(ws + p.acc);
  if (p.copy_w) {
    copy_rows(weight, weight_stride, vocab, width, ws + p.w, p.cs, s);
    w = (const uint16_t*)(ws + p.w);
    ldw = p.cs;
  }
  copy_rows_kernel<<<dim3((uint32_t)std::min<int64_t>(tokens, 8192) + 1), dim3(256), 0, s>>>(
      (const uint16_t*)hidden, hidden_stride, tokens, width, (uint16_t*)(ws + p.h), p.cs, targets,
      target_bytes, vocab, grad_loss, gmax);
  if (int rc = launched(who)) return rc;
  for (int64_t v0 = 0; v0 < vocab; v0 += p.piece) {
    const int64_t rows = std::min(p.piece, vocab - v0), cols = up(rows, 8);
    if (tokens) {
      GemmArgs a{};
      shape(&a, p.small, rows, tokens, p.wp, 1);
      a.a = w + v0 * ldw;
      a.lda = ldw;
      a.b = h;
      a.ldb = p.cs;
      a.targets = targets;
      a.target_bytes = target_bytes;
      a.vocab = vocab;
      a.v0 = v0;
      a.lse = lse;
      a.gloss = grad_loss;
      a.gmax = gmax;
      a.g = g;
      a.ldg = cols;
      launch<kGrad, kByK, kByK>(a, p.small, dtype, 1, s);
    }
    if (grad_weight) {
      GemmArgs a{};
      shape(&a, p.small_w, width, rows, tokens, 1);
      a.a = h;
      a.lda = p.cs;
      a.b = g;
      a.ldb = cols;
      a.gmax = gmax;
      a.c = (uint16_t*)grad_weight + v0 * grad_weight_stride;
      a.ldc = grad_weight_stride;
      a.c_wide = wide(grad_weight, grad_weight_stride, dtype);
      launch<kStore, kByRow, kByRow>(a, p.small_w, dtype, 1, s);
    }
    if (grad_hidden && tokens) {
      GemmArgs a{};
      shape(&a, p.small_h, width, tokens, rows, p.splits);
      a.a = w + v0 * ldw;
      a.lda = ldw;
      a.b = g;
      a.ldb = cols;
      a.acc = acc;
      a.ldc = p.wp;
      a.acc_split = tokens * p.wp;
      a.add = v0 > 0;
      launch<kAccum, kByRow, kByK>(a, p.small_h, dtype, p.splits, s);
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
