// embed.hip -- the token embedding and its table's gradient.
//
// Forward: out[t] = scale * table[id_t].  A copy of T rows: bound by the bytes
// (the rows read and written); a lane moves 8 elements, a row takes the least
// power of two of lanes that covers it, up to a workgroup.  16384 tokens of 4096 bf16:
// 33 us for 268 MB read and written (8 TB/s: frequent ids' rows come from the caches).
//
// Backward: grad_table[v] = scale * sum over {t : id_t = v} of grad_out[t].
// Frequencies of a language fall as one over the rank: some ids own a tenth of
// all tokens, most none.  Atomics would make the sum's order a matter of
// timing, so tokens are grouped by id first:
//   sort_kernel    one workgroup per bucket of ids (id mod the power-of-two
//                  number of buckets, so that neighbouring frequent ids part).
//                  It reads all ids, counts its own per id and wave, and places
//                  them in order of t; the tokens of lower buckets, counted
//                  along the way, give its place in the output.  One launch, no
//                  exchange between workgroups.  T ids are read by every bucket
//                  twice, out of L2.
//   reduce_kernel  fixed runs of 8 or 32 sorted tokens, a wave per run and 512
//                  columns: the rows of one id are summed in fp32 in order.  An
//                  id whose tokens lie in one run is written at once; of one that
//                  crosses runs, each run stores its part in fp32.  Waves of
//                  the same launch write the zero rows of ids without tokens.
//   join_kernel    adds the parts of an id that crosses runs, in their order.
// The work is balanced by tokens, not ids, and the order is fixed.  Bound by HBM: the
// gradient's rows read and the table written.  16384 tokens, 32000 x 4096 bf16:
// a call of 94 us for 396 MB (4.2 TB/s), its kernels 12 + 66 + 7.  Small calls are bound by
// the three launches' chain: 3001 tokens, 32003 x 1001 fp16 in 23.5 us, 9 + 12 + 4.
#include <algorithm>

#include "ops.h"

namespace zs {
namespace ops {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kBatch = 16;       // ids that a lane holds
constexpr int kMaxSlots = 512;   // ids of one bucket
constexpr int kMaxRun = 32;      // sorted tokens of one wave at most
constexpr int kAhead = 8;        // of whose rows are on their way at a time
constexpr int kCols = 512;       // columns of one wave
constexpr int kJoin = 16;        // parts that are read together

// A run's last id, where it begins in the run and goes on, and the run it ends in.
struct Crossing {
  int32_t id, last_run;  // id -1: none
};

template <typename I>
__device__ __forceinline__ int64_t local_id(const void* ids, int64_t t, int64_t start) {
  return (int64_t)((const I*)ids)[t] - start;
}

template <int DT, typename I>
__global__ __launch_bounds__(256) void gather_kernel(
    const elem_t<DT>* __restrict__ table, int64_t table_stride, const void* __restrict__ ids,
    elem_t<DT>* __restrict__ out, int64_t out_stride, int64_t n, int64_t vocab, int64_t width,
    int64_t start, float scale, int lanes_log2) {
  const int lanes = 1 << lanes_log2;
  const int64_t t = ((int64_t)blockIdx.x << (8 - lanes_log2)) + (threadIdx.x >> lanes_log2);
  if (t >= n) return;
  const int64_t v = local_id<I>(ids, t, start);
  const bool in = v >= 0 && v < vocab;
  const elem_t<DT>* src = table + (in ? v : 0) * table_stride;
  elem_t<DT>* dst = out + t * out_stride;
  for (int64_t c = (int64_t)(threadIdx.x & (lanes - 1)) * 8; c < width; c += lanes * 8) {
    f32x8 x = {};
    if (in) x = load8<DT>(src + c, width - c) * scale;
    store8<DT>(dst + c, width - c, x);
  }
}

template <typename I>
__global__ __launch_bounds__(kSortThreads) void sort_kernel(
    const void* __restrict__ ids, int32_t n, int64_t vocab, int64_t start, int bucket_log2,
    int32_t* __restrict__ order, int32_t* __restrict__ sorted, int32_t* __restrict__ first,
    int32_t* __restrict__ count, int32_t* __restrict__ n_valid) {
  __shared__ int32_t cnt[kSortWaves][kMaxSlots];
  __shared__ int32_t scan[kSortWaves];
  __shared__ int32_t lower;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t bucket = blockIdx.x, buckets = 1u << bucket_log2;
  const int slots = (int)((vocab + buckets - 1) >> bucket_log2);
  for (int i = threadIdx.x; i < slots; i += kSortThreads)
#pragma unroll
    for (int w = 0; w < kSortWaves; w++) cnt[w][i] = 0;
  if (threadIdx.x == 0) lower = 0;
  __syncthreads();
  // each wave has a stretch of the tokens, a multiple of 64, and takes kBatch
  // loads of it at a time; a stretch of one batch stays in registers
  const int64_t per = ((int64_t)n + kSortThreads - 1) / kSortThreads * 64;
  const int64_t begin = wave * per, end = begin + per < n ? begin + per : n;
  int32_t held[kBatch];
  auto load = [&](int64_t t0) {
#pragma unroll
    for (int i = 0; i < kBatch; i++) {
      const int64_t t = t0 + i * 64 + lane;
      // past the end the last id is read again, so that all loads go out at once
      const int64_t v = local_id<I>(ids, t < end ? t : end - 1, start);
      held[i] = t < end && v >= 0 && v < vocab ? (int32_t)v : -1;
    }
  };
  int32_t less = 0;
  for (int64_t t0 = begin; t0 < end; t0 += kBatch * 64) {
    load(t0);
#pragma unroll
    for (int i = 0; i < kBatch; i++) {
      const uint32_t b = (uint32_t)held[i] & (buckets - 1);
      if (held[i] < 0) continue;
      less += b < bucket;
      if (b == bucket) atomicAdd(&cnt[wave][(uint32_t)held[i] >> bucket_log2], 1);
    }
  }
  for (int d = 1; d < 64; d <<= 1) less += __shfl_xor(less, d, 64);
  if (lane == 0 && less) atomicAdd(&lower, less);
  __syncthreads();
  // a thread per id: its tokens before each wave, and all ids' before it
  const bool owner = (int)threadIdx.x < slots;
  int32_t total = 0, before[kSortWaves];
#pragma unroll
  for (int w = 0; w < kSortWaves; w++) before[w] = owner ? cnt[w][threadIdx.x] : 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; w++) {
    const int32_t c = before[w];
    before[w] = total;
    total += c;
  }
  int32_t upto = total;
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t o = __shfl_up(upto, d, 64);
    if (lane >= d) upto += o;
  }
  if (lane == 63) scan[wave] = upto;
  __syncthreads();
  int32_t at = lower + upto - total;
  for (int w = 0; w < wave; w++) at += scan[w];
  if (owner) {
#pragma unroll
    for (int w = 0; w < kSortWaves; w++) cnt[w][threadIdx.x] = at + before[w];
    const int64_t v = ((int64_t)threadIdx.x << bucket_log2) + bucket;
    if (v < vocab) {
      first[v] = at;
      count[v] = total;
    }
  }
  if (bucket == buckets - 1 && threadIdx.x == kSortThreads - 1) *n_valid = at + total;
  __syncthreads();
  for (int64_t t0 = begin; t0 < end; t0 += kBatch * 64) {
    if (per > kBatch * 64) load(t0);
#pragma unroll
    for (int i = 0; i < kBatch; i++) {
      const bool mine = held[i] >= 0 && ((uint32_t)held[i] & (buckets - 1)) == bucket;
      const int32_t slot = held[i] >> bucket_log2;
      uint64_t todo = __ballot(mine);
      while (todo) {  // one id of these 64 tokens at a time, its tokens in order
        const int leader = __builtin_ctzll(todo);
        const int32_t s = __builtin_amdgcn_readlane(slot, leader);
        const bool same = mine && slot == s;
        const uint64_t peers = __ballot(same);
        // one lane takes the places of all: no lane reads what another wrote
        int32_t first_place = 0;
        if (lane == leader)
          first_place = atomicAdd(&cnt[wave][s], (int32_t)__builtin_popcountll(peers));
        first_place = __builtin_amdgcn_readlane(first_place, leader);
        if (same) {
          const int32_t place =
              first_place + (int32_t)__builtin_popcountll(peers & ((1ull << lane) - 1));
          order[place] = (int32_t)(t0 + i * 64 + lane);
          sorted[place] = held[i];
        }
        todo &= ~peers;
      }
    }
  }
}

template <int TT, bool NT>
__device__ __forceinline__ void put_row(elem_t<TT>* p, int64_t n, f32x8 sum, float scale,
                                        bool add) {
  f32x8 x = sum * scale;
  if (add) x += load8<TT>(p, n);
  store8<TT, NT>(p, n, x);
}

// Zeros to n elements at p by a wave: aligned 16-byte pieces, and the elements before
// and after them one by one.  Rows of an odd width start anywhere, and streamed
// stores that leave lines half written cost twice the time (308 tokens, 38364 x
// 6997 fp32: 505 us with a wave a 512-column slab at the row's own alignment).
template <int TT, bool NT>
__device__ __forceinline__ void zero_row(elem_t<TT>* p, int64_t n, int lane) {
  constexpr int kPer = 16 / (int)sizeof(elem_t<TT>);
  const int64_t skew = (int64_t)((uintptr_t)p / sizeof(elem_t<TT>)) & (kPer - 1);
  int64_t head = skew ? kPer - skew : 0;
  if (head > n) head = n;
  const int64_t whole = (n - head) / kPer, tail = head + whole * kPer;
  if (lane < head) p[lane] = (elem_t<TT>)0.0f;
  for (int64_t i = lane; i < whole; i += 64) st16<NT>(p + head + i * kPer, u32x4{});
  if (tail + lane < n) p[tail + lane] = (elem_t<TT>)0.0f;
}

template <int DT, int TT, bool NT>
__global__ __launch_bounds__(256) void reduce_kernel(
    const elem_t<DT>* __restrict__ grad, int64_t grad_stride, elem_t<TT>* __restrict__ table,
    int64_t table_stride, int64_t vocab, int64_t width, float scale, int accumulate,
    const int32_t* __restrict__ order, const int32_t* __restrict__ sorted,
    const int32_t* __restrict__ first, const int32_t* __restrict__ count,
    const int32_t* __restrict__ n_valid, float* __restrict__ parts, int64_t part_stride,
    Crossing* __restrict__ crossings, int64_t run_items, int64_t slabs, int run, int zero_rows) {
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t unit = item / slabs;
  const int64_t c = (item - unit * slabs) * kCols + lane * 8;
  const int64_t left = width - c;
  if (unit >= run_items) {  // ids without tokens, zero_rows whole rows a wave
    if (accumulate) return;
    const int64_t v0 = (item - run_items * slabs) * zero_rows;
    for (int64_t v = v0; v < v0 + zero_rows && v < vocab; v++)
      if (count[v] == 0) zero_row<TT, NT>(table + v * table_stride, width, lane);
    return;
  }
  const int64_t valid = *n_valid;
  const int64_t p0 = unit * run;
  const int n = (int)(valid - p0 < run ? valid - p0 : run);
  if (n <= 0) {
    if (c == 0) crossings[unit] = {-1, 0};
    return;
  }
  const int64_t mine = p0 + (lane < n ? lane : n - 1);
  const int32_t my_t = order[mine], my_v = sorted[mine];
  const int32_t my_first = first[my_v], my_count = count[my_v];
  if (c - lane * 8 == 0 && lane == n - 1) {  // the last token's id: does it begin here and go on?
    const int64_t end = (int64_t)my_first + my_count;
    const bool goes_on = my_first >= p0 && end > p0 + n;
    crossings[unit] = {goes_on ? my_v : -1, (int32_t)((end - 1) / run)};
  }
  f32x8 sum = {};
  for (int i = 0; i < n; i += kAhead) {
    Chunk<DT> x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; j++) {
      const int k = i + j < n ? i + j : n - 1;
      const int64_t t = __builtin_amdgcn_readlane(my_t, k);
      x[j] = load_row<DT>(grad + t * grad_stride, c, width);
    }
#pragma unroll
    for (int j = 0; j < kAhead; j++) {
      if (i + j >= n) break;
      sum += take8<DT>(x[j], left, width);
      const int64_t b = __builtin_amdgcn_readlane(my_first, i + j);
      const int64_t e = b + __builtin_amdgcn_readlane(my_count, i + j);
      const int64_t next = p0 + i + j + 1;
      if (next != e && i + j + 1 < n) continue;
      if (left > 0) {  // the id's last token, or the run's
        if (b >= p0 && next == e) {
          const int64_t v = __builtin_amdgcn_readlane(my_v, i + j);
          put_row<TT, NT>(table + v * table_stride + c, left, sum, scale, accumulate != 0);
        } else {  // slot 0: the id came from the run before; slot 1: it begins here
          float* part = parts + (unit * 2 + (b >= p0)) * part_stride + c;
          store8<ZS_F32>(part, 8, sum);
        }
      }
      sum = f32x8{};
    }
  }
}

template <int TT>
__global__ __launch_bounds__(256) void join_kernel(
    elem_t<TT>* __restrict__ table, int64_t table_stride, int64_t width, float scale,
    int accumulate, const Crossing* __restrict__ crossings, const float* __restrict__ parts,
    int64_t part_stride, int64_t run_items, int64_t slabs) {
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t unit = item / slabs;
  const int64_t c = (item - unit * slabs) * kCols + lane * 8;
  if (unit >= run_items) return;
  const Crossing crossing = crossings[unit];
  const int64_t left = width - c;
  if (crossing.id < 0 || left <= 0) return;
  const int64_t end = crossing.last_run;
  f32x8 sum = load8<ZS_F32>(parts + (unit * 2 + 1) * part_stride + c, 8);
  int64_t r = unit + 1;
  for (; r <= end; r += kJoin) {  // so many parts on their way at a time
    f32x8 x[kJoin];
#pragma unroll
    for (int j = 0; j < kJoin; j++)
      x[j] = load8<ZS_F32>(parts + (r + j) * 2 * part_stride + c, r + j <= end ? 8 : 0);
#pragma unroll
    for (int j = 0; j < kJoin; j++)
      if (r + j <= end) sum += x[j];
  }
  put_row<TT, false>(table + (int64_t)crossing.id * table_stride + c, left, sum, scale, accumulate != 0);
}

struct Layout {
  int bucket_log2, run;
  int64_t runs, slabs, part_stride;
  size_t order, sorted, first, count, n_valid, crossings, parts, total;
};
constexpr int64_t kMaxVocab = 1 << 24, kMaxTokens = 0x7fffffff;

Layout layout(int64_t n, int64_t vocab, int64_t width) {
  Layout l{};
  l.bucket_log2 = 8;
  while (((vocab + (1ll << l.bucket_log2) - 1) >> l.bucket_log2) > kMaxSlots) l.bucket_log2++;
  l.slabs = (width + kCols - 1) / kCols;
  // short runs where there are few wave-rows (tokens times slabs), since a wave's rows come one
  // batch after another; long ones where there are more, with fewer parts to join.  Runs of
  // 8 and of 32, the call's us: 3001 tokens of 1001 23 and 32, 6000 of 1001 28 and 32, 8192 of
  // 512 26 and 29; about equal at 12000 wave-rows (12000 of 512 30 and 30, 1500 of 4096 60 and
  // 58); 4096 of 4096 69 and 59, 16384 of 1024 41 and 35, 60000 of 512 96 and 70.
  l.run = n * l.slabs <= 12288 ? 8 : kMaxRun;
  l.runs = (n + l.run - 1) / l.run;
  l.part_stride = (width + 7) / 8 * 8;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at += up256(bytes);
    return p;
  };
  l.order = take((size_t)n * 4);
  l.sorted = take((size_t)n * 4);
  l.first = take((size_t)vocab * 4);
  l.count = take((size_t)vocab * 4);
  l.n_valid = take(4);
  l.crossings = take((size_t)l.runs * sizeof(Crossing));
  l.parts = take((size_t)l.runs * 2 * l.part_stride * 4);
  l.total = at;
  return l;
}

constexpr int64_t kMaxWidth = 1 << 20, kMaxBlocks = 0x7fffff;  // 2^31 lanes of a launch

int check_ids(const char* who, const void* ids, int64_t n, int64_t vocab, int64_t width,
              int32_t id_bytes, float scale) {
  if (n < 0 || vocab < 1 || vocab > kMaxVocab || width < 1 || width > kMaxWidth ||
      n > kMaxTokens)
    return fail(who, "a size is out of range");
  if (id_bytes != 4 && id_bytes != 8) return fail(who, "ids are 4 or 8 bytes");
  if (n && !ids) return fail(who, "ids is NULL");
  if (!al(ids, id_bytes)) return fail(who, "ids are not aligned to their size");
  if (!__builtin_isfinite(scale)) return fail(who, "scale must be finite");
  return ZS_OK;
}

}  // namespace
}  // namespace ops
}  // namespace zs

using namespace zs::ops;

extern "C" int zs_embed_forward(const void* table, int64_t table_stride, const void* ids,
                                void* out, int64_t out_stride, int64_t n_tokens, int64_t vocab,
                                int64_t width, int64_t vocab_start, float scale, int32_t dtype,
                                int32_t id_bytes, void* stream) {
  const char* who = "zs_embed_forward";
  if (!good_dtype(dtype)) return fail(who, "unknown element type");
  if (int rc = check_ids(who, ids, n_tokens, vocab, width, id_bytes, scale)) return rc;
  if (table_stride < width || out_stride < width) return fail(who, "a row stride is below width");
  if (n_tokens == 0) return ZS_OK;
  if (!table || !out) return fail(who, "NULL buffer");
  if (!al(table, elem_bytes(dtype)) || !al(out, elem_bytes(dtype)))
    return fail(who, "a buffer is not aligned to its elements");
  int log2 = 3;
  while (log2 < 8 && (8ll << log2) < width) log2++;
  const int64_t blocks = (n_tokens + (256 >> log2) - 1) >> (8 - log2);
  if (blocks > kMaxBlocks) return fail(who, "too many tokens for one call");
  with_dtype(dtype, [&](auto DT) {
    with_bool(id_bytes == 8, [&](auto I8) {
      using E = elem_t<decltype(DT)::value>;
      using I = std::conditional_t<decltype(I8)::value, int64_t, int32_t>;
      gather_kernel<decltype(DT)::value, I>
          <<<dim3((uint32_t)blocks), dim3(256), 0, (hipStream_t)stream>>>(
              (const E*)table, table_stride, ids, (E*)out, out_stride, n_tokens, vocab, width,
              vocab_start, scale, log2);
    });
  });
  return launched(who);
}

extern "C" size_t zs_embed_backward_bytes(int64_t n_tokens, int64_t vocab, int64_t width) {
  if (n_tokens < 0 || n_tokens > kMaxTokens || vocab < 1 || vocab > kMaxVocab || width < 1 ||
      width > kMaxWidth)
    return 0;
  return layout(n_tokens, vocab, width).total;
}

extern "C" int zs_embed_backward(const void* grad_out, int64_t grad_stride, const void* ids,
                                 void* grad_table, int64_t table_stride, int64_t n_tokens,
                                 int64_t vocab, int64_t width, int64_t vocab_start, float scale,
                                 int32_t dtype, int32_t table_dtype, int32_t id_bytes,
                                 int32_t accumulate, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  const char* who = "zs_embed_backward";
  if (!good_dtype(dtype)) return fail(who, "unknown element type");
  if (table_dtype != dtype && table_dtype != ZS_F32)
    return fail(who, "the table's gradient has the gradient's type or fp32");
  if (int rc = check_ids(who, ids, n_tokens, vocab, width, id_bytes, scale)) return rc;
  if (table_stride < width || grad_stride < width)
    return fail(who, "a row stride is below width");
  if (!grad_table || (n_tokens && !grad_out)) return fail(who, "NULL buffer");
  if (!al(grad_table, elem_bytes(table_dtype)) || !al(grad_out, elem_bytes(dtype)))
    return fail(who, "a buffer is not aligned to its elements");
  const Layout l = layout(n_tokens, vocab, width);
  if (!workspace || !al(workspace, 256)) return fail(who, "the workspace is NULL or not 256-byte aligned");
  if (workspace_bytes < l.total) return fail(who, "the workspace is too small");
  // rows without tokens of about 4 KB a wave
  const int zero_rows =
      (int)std::min<int64_t>(8, std::max<int64_t>(1, 4096 / (width * elem_bytes(table_dtype))));
  const int64_t zero_items = accumulate ? 0 : (vocab + zero_rows - 1) / zero_rows;
  const int64_t blocks = (l.runs * l.slabs + zero_items + 3) / 4;
  const int64_t join_blocks = (l.runs * l.slabs + 3) / 4;
  if (blocks > kMaxBlocks) return fail(who, "too many rows for one call");
  if (blocks == 0) return ZS_OK;  // no tokens to add
  uint8_t* ws = (uint8_t*)workspace;
  int32_t *order = (int32_t*)(ws + l.order), *sorted = (int32_t*)(ws + l.sorted),
          *first = (int32_t*)(ws + l.first), *count = (int32_t*)(ws + l.count),
          *n_valid = (int32_t*)(ws + l.n_valid);
  float* parts = (float*)(ws + l.parts);
  Crossing* crossings = (Crossing*)(ws + l.crossings);
  hipStream_t s = (hipStream_t)stream;
  with_bool(id_bytes == 8, [&](auto I8) {
    using I = std::conditional_t<decltype(I8)::value, int64_t, int32_t>;
    sort_kernel<I><<<dim3(1u << l.bucket_log2), dim3(kSortThreads), 0, s>>>(
        ids, (int32_t)n_tokens, vocab, vocab_start, l.bucket_log2, order, sorted, first, count,
        n_valid);
  });
  if (int rc = launched(who)) return rc;
  const bool nt = streams((n_tokens * elem_bytes(dtype) + vocab * elem_bytes(table_dtype)) * width);
  auto go = [&](auto DT, auto TT) {
    using E = elem_t<decltype(DT)::value>;
    using T = elem_t<decltype(TT)::value>;
    with_bool(nt, [&](auto NT) {
      reduce_kernel<decltype(DT)::value, decltype(TT)::value, decltype(NT)::value>
          <<<dim3((uint32_t)blocks), dim3(256), 0, s>>>(
              (const E*)grad_out, grad_stride, (T*)grad_table, table_stride, vocab, width, scale,
              accumulate, order, sorted, first, count, n_valid, parts, l.part_stride, crossings,
              l.runs, l.slabs, l.run, zero_rows);
    });
    if (l.runs > 1)
      join_kernel<decltype(TT)::value><<<dim3((uint32_t)join_blocks), dim3(256), 0, s>>>(
          (T*)grad_table, table_stride, width, scale, accumulate, crossings, parts, l.part_stride,
          l.runs, l.slabs);
  };
  if (table_dtype == dtype)
    with_dtype(dtype, [&](auto DT) { go(DT, DT); });
  else
    with_dtype(dtype, [&](auto DT) { go(DT, std::integral_constant<int, ZS_F32>()); });
  return launched(who);
}
