// mx4.hip -- matrices in 4 bits with a scale for each 32 neighbours, and their product.
//
// Packing: a group's scale is the least power of two that brings it within 6, its codes the
// elements over that scale rounded to {0, 1/2, 1, 3/2, 2, 3, 4, 6}, ties to even: 17 bytes for 32
// elements.  Bound by HBM.  Along rows a lane has 8 elements and a group's maximum is one over
// 4 neighbouring lanes.  Along columns (the transpose's rows) a tile of 128 x 128 goes through
// LDS and a lane takes 32 rows of two columns; with both wanted the tile is read once.
//
// The product: out[t][n] = sum_k x[t][k] w[n][k] of the values codes * scales, on 16x16x128
// matrix instructions that take the scales themselves (4-bit in, fp32 sums), one rounding at
// the end.  A lane of an instruction has one row's group of 32: 16 bytes of codes and a
// byte of a register that holds the scales of four instructions; the scales lie in memory in
// just that order (scale4_at), so that they go the codes' way with no rearrangement.
//
// Tiles of 256 features x 128 tokens, four waves of 128 x 64: a wave's 128 sums a lane leave room
// for a second workgroup on the compute unit, whose products run while this one waits, reads
// or writes its tile.  128 k a step, three steps in LDS, which global memory is read straight
// into.  A row's 64 bytes hold chunk c at c ^ ((row >> 2) & 3), so that the 8 rows that are
// read at a time lie on different banks.  Rows past the edge and groups past the end read as
// zeros by the buffer loads' bounds check.
//
// Few tokens: the weight is what is read, each of its rows by one workgroup, whose waves share
// k out between them and add their sums in LDS.
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

// A tile of 128 x 128: its rows' groups where ROWS, and its columns'.
template <int DT, bool ROWS>
__global__ __launch_bounds__(256) void pack_tile_kernel(
    const elem_t<DT>* __restrict__ x, int64_t x_stride, uint8_t* __restrict__ codes,
    uint8_t* __restrict__ scales, uint8_t* __restrict__ codes_t, uint8_t* __restrict__ scales_t,
    int64_t rows, int64_t width, uint32_t tiles_down) {
  typedef elem_t<DT> pair_t __attribute__((ext_vector_type(2)));
  __shared__ __attribute__((aligned(16))) elem_t<DT> tile[128][128];
  const int64_t r0 = (int64_t)(blockIdx.x % tiles_down) * 128;
  const int64_t c0 = (int64_t)(blockIdx.x / tiles_down) * 128;
  const int tid = threadIdx.x;
  const int64_t groups = groups_of(width), groups_t = groups_of(rows);
  Chunk<DT> in[8];
#pragma unroll
  for (int k = 0; k < 8; k++) {
    const int64_t row = r0 + (tid >> 4) + k * 16, c = c0 + (tid & 15) * 8;
    in[k] = Chunk<DT>{};
    if (row < rows && c < width) in[k] = load_chunk<DT>(x + row * x_stride + c, width - c);
  }
#pragma unroll
  for (int k = 0; k < 8; k++) {
    const int r = (tid >> 4) + k * 16, chunk = tid & 15;
    *(Chunk<DT>*)&tile[r][chunk * 8] = in[k];
    if (ROWS) {
      const f32x8 v = widen<DT>(in[k]);
      uint32_t byte;
      const uint32_t w = quantise4(v, group_amax(v, 4), &byte);
      const int64_t row = r0 + r, group = c0 / 32 + (chunk >> 2);
      if (row < rows) {
        if (group < groups) *(uint32_t*)(codes + row * groups * 16 + c0 / 2 + chunk * 4) = w;
        if ((chunk & 3) == 0)
          scales[scale4_at(row, group, rows)] = (uint8_t)(group < groups ? byte : 127u);
      }
    }
  }
  __syncthreads();
  const int lane = tid & 63, wave = tid >> 6;
  pair_t p[32];
#pragma unroll
  for (int i = 0; i < 32; i++) p[i] = *(const pair_t*)&tile[wave * 32 + i][lane * 2];
  const int64_t group = r0 / 32 + wave;
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const int64_t col = c0 + lane * 2 + h;
    if (col >= width) return;
    f32x8 v[4];
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 4; q++) {
#pragma unroll
      for (int i = 0; i < 8; i++) v[q][i] = (float)p[q * 8 + i][h];
      const uint32_t a = amax_bits(v[q]);
      m = a > m ? a : m;
    }
    u32x4 w;
    uint32_t byte;
#pragma unroll
    for (int q = 0; q < 4; q++) w[q] = quantise4(v[q], __uint_as_float(m), &byte);
    if (group < groups_t) *(u32x4*)(codes_t + (col * groups_t + group) * 16) = w;
    scales_t[scale4_at(col, group, width)] = (uint8_t)(group < groups_t ? byte : 127u);
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

struct Mx4Args {
  const uint8_t *a, *b;    // codes of w (features) and x (tokens)
  const uint8_t *as, *bs;  // scales
  int64_t m, n;            // features, tokens
  int32_t groups;          // of k
  int32_t tiles_m, tiles_n;
  void* c;
  int64_t ldc;
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

// R rows of an operand: their way from memory to LDS, 64 bytes of codes a step and 16 of scales
// a span of four steps.
template <int R>
struct Side {
  static constexpr int kLoads = R * 64 / 4096;  // of a thread, for a step
  const uint8_t* codes;  // the tile's first row
  const uint8_t* scales;
  int64_t ld, span;      // bytes of a row, and of a span's scales
  int32_t rows, groups;
  uint32_t off[kLoads];
  int32_t chunk;

  __device__ __forceinline__ Side(const uint8_t* c, const uint8_t* s, int64_t row0, int64_t n,
                                  int32_t g, int tid) {
    ld = (int64_t)g * 16;
    span = n * 16;
    codes = c + row0 * ld;
    scales = s + row0 * 16;
    rows = (int32_t)(n - row0 < R ? n - row0 : R);
    groups = g;
    const int row = tid >> 2;
    chunk = (tid & 3) ^ ((row >> 2) & 3);  // 64 rows on, the same
#pragma unroll
    for (int i = 0; i < kLoads; i++) off[i] = (uint32_t)((row + i * 64) * ld + chunk * 16);
  }
  // The codes of a step, into LDS at `lds` (the wave's part of the first load).  Groups past the
  // end would be the next row's: there a lane reads out of bounds.
  __device__ __forceinline__ void load(int step, uint32_t lds) {
    const int32_t left = groups - step * 4;
    if (left < 4) {
#pragma unroll
      for (int i = 0; i < kLoads; i++) off[i] = chunk < left ? off[i] : 0xfffffff0u;
    }
    const u32x4 d = descriptor(codes + step * 64, left > 0 ? (rows - 1) * ld + left * 16 : 0);
#pragma unroll
    for (int i = 0; i < kLoads; i++) load_lds(d, off[i], lds + i * 4096);
  }
};

// What lane `lane` has of fragment f of a step's rows.
__device__ __forceinline__ i32x4 fragment(const uint8_t* tile, int row0, int f, int lane) {
  const int row = row0 + (lane & 15);
  return *(const i32x4*)(tile + row * 64 + (((lane >> 4) ^ ((row >> 2) & 3)) * 16) + f * 1024);
}

template <int DT, int BM, int BN>
__global__ __launch_bounds__(256, 2) void product_kernel(Mx4Args g) {
  constexpr int FM = BM / 32, FN = BN / 32;  // fragments of a wave: two waves by two
  constexpr int kTile = (BM + BN) * 64, kScales = (BM + BN) * 16;
  constexpr int kLoads = Side<BM>::kLoads + Side<BN>::kLoads;
  constexpr int kScaleLoads = (kScales + 4095) / 4096;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[3 * kTile + kScaleLoads * 4096];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int32_t tm, tn;
  tile_of(g, &tm, &tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int steps = (g.groups + 3) / 4;
  Side<BM> a(g.a, g.as, m0, g.m, g.groups, tid);
  Side<BN> b(g.b, g.bs, n0, g.n, g.groups, tid);
  const uint32_t lds_at = (uint32_t)(uintptr_t)(ZS_LDS uint8_t*)lds + wave * 1024;
  uint8_t* const scale_tile = lds + 3 * kTile;

  // The scales of span p: a load of a thread is 16 bytes, those of one row.
  auto load_scales = [&](int p) {
    const bool there = p * 4 < steps;
    const u32x4 da = descriptor(a.scales + p * a.span, there ? a.rows * 16 : 0);
    const u32x4 db = descriptor(b.scales + p * b.span, there ? b.rows * 16 : 0);
#pragma unroll
    for (int i = 0; i < kScaleLoads; i++) {
      // A's rows and then B's; BM is whole waves' rows
      const int row = i * 256 + wave * 64;
      const uint32_t to = lds_at + 3 * kTile + i * 4096;
      if (row < BM)
        load_lds(da, (uint32_t)((row + lane) * 16), to);
      else
        load_lds(db, (uint32_t)((row - BM + lane) * 16), to);
    }
  };
  auto load = [&](int step, int stage) {
    a.load(step, lds_at + stage * kTile);
    b.load(step, lds_at + stage * kTile + BM * 64);
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
  load(1, 1);
  int stage = 0;
  // Step `step`, the J-th of its span.  Its codes have landed for every wave, and every
  // wave has read the step before, whose place takes the loads of the step after next.
  auto one = [&](auto J, int step) {
    constexpr int j = decltype(J)::value;
    // what may still be on its way: the next step's codes and, after them, a span's scales
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(
                     j == 2 ? kLoads + kScaleLoads : kLoads)
                 : "memory");
    const uint8_t* tile = lds + stage * kTile;
    if (j == 0) {
#pragma unroll
      for (int i = 0; i < FM; i++)
        sa[i] = *(const uint32_t*)(scale_tile + (ra + i * 16 + (lane & 15)) * 16 + (lane >> 4) * 4);
#pragma unroll
      for (int i = 0; i < FN; i++)
        sb[i] = *(const uint32_t*)(scale_tile + (BM + rb + i * 16 + (lane & 15)) * 16 + (lane >> 4) * 4);
    }
    i32x4 fb[FN];
#pragma unroll
    for (int i = 0; i < FN; i++) fb[i] = fragment(tile + BM * 64, rb, i, lane);
    const int ahead = stage == 0 ? 2 : stage - 1;
    if (j == 1) load_scales((step >> 2) + 1);
    load(step + 2, ahead);
#pragma unroll
    for (int i = 0; i < FM; i++) {
      const i32x4 fa = fragment(tile, ra, i, lane);
#pragma unroll
      for (int k = 0; k < FN; k++) acc[i][k] = mfma4<j>(fa, fb[k], acc[i][k], sa[i], sb[k]);
    }
    stage = stage == 2 ? 0 : stage + 1;
  };
  for (int step = 0; step < steps; step += 4) {
    one(std::integral_constant<int, 0>(), step);
    if (step + 1 < steps) one(std::integral_constant<int, 1>(), step + 1);
    if (step + 2 < steps) one(std::integral_constant<int, 2>(), step + 2);
    if (step + 3 < steps) one(std::integral_constant<int, 3>(), step + 3);
  }
  // no load is on its way into LDS any more
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  // acc[i][k][r]: feature m0 + ra + i*16 + (lane>>4)*4 + r, token n0 + rb + k*16 + (lane&15)
#pragma unroll
  for (int k = 0; k < FN; k++) {
    const int64_t t = n0 + rb + k * 16 + (lane & 15);
    if (t >= g.n) continue;
    elem_t<DT>* row = (elem_t<DT>*)g.c + t * g.ldc;
#pragma unroll
    for (int i = 0; i < FM; i++) {
      const int64_t f = m0 + ra + i * 16 + (lane >> 4) * 4;
      if (f < g.m) store4<DT>(row + f, g.m - f, acc[i][k]);
    }
  }
}

// Few tokens: 32 features a workgroup, FN * 16 tokens, spans of k dealt out over eight waves.
constexpr int kFewWaves = 8;
template <int DT, int FN>
__global__ __launch_bounds__(kFewWaves * 64) void few_kernel(Mx4Args g) {
  constexpr int FM = 2;
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
  for (int p = wave; p < spans; p += kFewWaves) {
    i32x4 fa[FM][4], fb[FN][4];
    uint32_t sa[FM], sb[FN];
    // rows that do not exist are the last one's, and go nowhere; groups past the end are zeros
    auto read = [&](const uint8_t* codes, const uint8_t* scales, int64_t row, int64_t rows,
                    i32x4(&f)[4], uint32_t& s) {
      row = row < rows ? row : rows - 1;
      s = *(const uint32_t*)(scales + ((int64_t)p * rows + row) * 16 + (lane >> 4) * 4);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int group = p * 16 + j * 4 + (lane >> 4);
        f[j] = i32x4{};
        if (group < g.groups) f[j] = *(const i32x4*)(codes + row * ld + group * 16);
      }
    };
#pragma unroll
    for (int i = 0; i < FM; i++) read(g.a, g.as, m0 + i * 16 + (lane & 15), g.m, fa[i], sa[i]);
#pragma unroll
    for (int k = 0; k < FN; k++) read(g.b, g.bs, n0 + k * 16 + (lane & 15), g.n, fb[k], sb[k]);
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

// Up to so many tokens the weight is streamed.
constexpr int64_t kFewTokens = 64;

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
  // tiles past the end too: they write the scales of groups that fill a span up
  const int64_t down = spans_t * 4, across = (codes ? spans * 4 : (width + 127) / 128);
  if (down * across > 0xffffff) return fail(who, "too many elements for one call");
  with_dtype(dtype, [&](auto DT) {
    with_bool(codes != nullptr, [&](auto ROWS) {
      pack_tile_kernel<decltype(DT)::value, decltype(ROWS)::value>
          <<<dim3((uint32_t)(down * across)), dim3(256), 0, (hipStream_t)stream>>>(
              (const elem_t<decltype(DT)::value>*)x, x_stride, (uint8_t*)codes, (uint8_t*)scales,
              (uint8_t*)codes_t, (uint8_t*)scales_t, rows, width, (uint32_t)down);
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

extern "C" int zs_mx4_product(const void* x_codes, const void* x_scales, const void* w_codes,
                              const void* w_scales, void* out, int64_t out_stride, int64_t tokens,
                              int64_t features, int64_t width, int32_t dtype, void* stream) {
  const char* who = "zs_mx4_product";
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
  const hipStream_t st = (hipStream_t)stream;
  if (tokens <= kFewTokens) {
    const uint32_t blocks = (uint32_t)((features + 31) / 32);
    with_dtype(dtype, [&](auto DT) {
      constexpr int kDt = decltype(DT)::value;
      if (tokens <= 16)
        few_kernel<kDt, 1><<<dim3(blocks, 1), dim3(kFewWaves * 64), 0, st>>>(g);
      else if (tokens <= 32)
        few_kernel<kDt, 2><<<dim3(blocks, 1), dim3(kFewWaves * 64), 0, st>>>(g);
      else
        few_kernel<kDt, 2><<<dim3(blocks, 2), dim3(kFewWaves * 64), 0, st>>>(g);
    });
    return launched(who);
  }
  auto tiles = [&](int64_t bm, int64_t bn) {
    g.tiles_m = (int32_t)((features + bm - 1) / bm);
    g.tiles_n = (int32_t)((tokens + bn - 1) / bn);
    return (int64_t)g.tiles_m * g.tiles_n;
  };
  const bool small = tiles(256, 128) < 512;
  const int64_t total = small ? tiles(128, 64) : tiles(256, 128);
  if (total > 0xffffff) return fail(who, "too many tiles for one call");
  with_dtype(dtype, [&](auto DT) {
    if (small)
      product_kernel<decltype(DT)::value, 128, 64><<<dim3((uint32_t)total), dim3(256), 0, st>>>(g);
    else
      product_kernel<decltype(DT)::value, 256, 128><<<dim3((uint32_t)total), dim3(256), 0, st>>>(g);
  });
  return launched(who);
}
