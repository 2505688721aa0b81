// xent_plan.h -- how a cross entropy call is divided: copies, tiles of the products, pieces of
// the vocabulary, and its workspace.  Plain C++, so that the rules can be looked at without
// a device.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace zs {
namespace ops {
namespace xent {

// G of one piece: 256 MB.  Every piece past the first reads and writes grad_hidden's fp32
// sums once more (0.1 ms at 8192 tokens of 4096, two pieces of 16000 entries).
constexpr int64_t kPieceElems = 128ll << 20;
constexpr int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

inline bool needs_copy(const void* p, int64_t stride, int64_t width) {
  return (uintptr_t)p % 16 || stride % 8 || width % 8;
}

constexpr int64_t kCus = 256;
inline int64_t tiles(int64_t m, int64_t n, bool small) {
  return small ? up(m, 128) / 128 * (up(n, 64) / 64) : up(m, 256) / 256 * (up(n, 256) / 256);
}
// Whether a product takes the small tiles: where few rows of B leave a large one mostly
// empty, and where large ones leave much of the card idle.  Loss and gradients, us with small
// and with large tiles throughout (tokens x width x vocab): 512 x 1024 x 8000 74 and 138, 1024 x
// 2048 x 4000 111 and 190, 300 x 1536 x 20000 154 and 179, 768 x 512 x 16000 108 and 131; about
// equal at 1500 x 1024 x 8000, 192 tiles of the logits, 172 and 171 (161 as chosen here); 1500 x
// 2048 x 8000 275 and 226, 2048 x 2048 x 8000 345 and 259, 1003 x 1000 x 32003 422 and 319.
// Between 150 and 192 tiles either may win by a tenth or more.
inline bool few(int64_t m, int64_t n, int64_t splits) {
  return n <= 128 || tiles(m, n, false) * splits <= 192;
}

struct Plan {
  int64_t wp;         // width in whole chunks of 8
  int64_t cs;         // row stride of the copies: whole cache lines
  bool copy_h, copy_w;
  bool small, small_h, small_w;  // tiles of 128 x 64: for the logits, grad_hidden, grad_weight
  int64_t parts;      // partial statistics a token (forward)
  int64_t piece;      // vocabulary entries a piece (backward)
  int32_t splits;     // of k in the product for grad_hidden
  size_t h, w, pmax, psum, tlogit, gmax, g, acc, total;
};

inline Plan plan(const void* hidden, int64_t h_stride, const void* weight, int64_t w_stride,
                 int64_t tokens, int64_t vocab, int64_t width, bool backward) {
  Plan p{};
  p.wp = up(width, 8);
  p.cs = up(width, 64);
  // the backward pass reads a copy whose rows that do not count are zeros
  p.copy_h = backward || needs_copy(hidden, h_stride, width);
  p.copy_w = needs_copy(weight, w_stride, width);
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t q = at;
    at += (size_t)up(bytes, 256);
    return q;
  };
  if (p.copy_h) p.h = take(tokens * p.cs * 2);
  if (p.copy_w) p.w = take(vocab * p.cs * 2);
  if (!backward) {
    p.small = few(vocab, tokens, 1);
    p.parts = up(vocab, p.small ? 128 : 256) / (p.small ? 128 : 256);
    p.pmax = take(p.parts * tokens * 4);
    p.psum = take(p.parts * tokens * 4);
    p.tlogit = take(tokens * 4);
  } else {
    const int64_t t = std::max<int64_t>(tokens, 1);
    const int64_t most = std::max<int64_t>(kPieceElems / up(t, 64) / 256 * 256, 256);
    const int64_t pieces = (vocab + most - 1) / most;
    p.piece = up((vocab + pieces - 1) / pieces, 256);
    p.small = few(p.piece, tokens, 1);
    p.small_w = few(width, p.piece, 1);
    // few tokens leave few tiles of grad_hidden: the piece's entries are divided
    // until the tiles cover the card, each part at least 512 long
    auto splits = [&](bool small) {
      return std::max<int64_t>(1, std::min(kCus / tiles(width, t, small), p.piece / 512));
    };
    p.small_h = few(width, tokens, splits(false));
    p.splits = (int32_t)splits(p.small_h);
    p.gmax = take(4);
    p.g = take(tokens * p.piece * 2);
    p.acc = take(p.splits * tokens * p.wp * 4);
  }
  p.total = std::max<size_t>(at, 256);
  return p;
}

}  // namespace xent
}  // namespace ops
}  // namespace zs
