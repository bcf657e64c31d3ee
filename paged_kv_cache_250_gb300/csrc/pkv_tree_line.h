// pkv_tree_line.h -- how the tree kernel's work is cut into shares.  Needs no CUDA.
//
// A segment is (sequence, pair of 128-row tiles, KV head): the rows are the
// sequence's nodes times the g query heads of the KV head, 256 to a pair.  Its
// units are the blocks of 128 cached tokens.  The segments lie on one line,
// sequence by sequence, pair by pair, head by head, where a segment's start
// costs kTreeSeg and a block kTreeTwo, or kTreeOne where the pair's second tile
// is empty.  The line is cut into n equal shares, one per CTA; a unit belongs to
// the share that its first cost lies in.
#pragma once

#include "pkv_hd.h"

namespace pkv {

constexpr int kTreeRows = 128, kTreeTok = 128;  // rows of a tile, tokens of a block
constexpr int kTreeOne = 3, kTreeTwo = 5, kTreeSeg = 4;
constexpr int kTreeMinShare = 8;  // a share is worth at least this much
constexpr int kTreeMaxBatch = 4000;

PKV_HD int tree_blocks(int ctx) { return (int)(((int64_t)ctx + kTreeTok - 1) / kTreeTok); }
PKV_HD int tree_pairs(int rows) { return (rows + 2 * kTreeRows - 1) / (2 * kTreeRows); }
PKV_HD bool tree_two(int rows, int pair) { return rows > (2 * pair + 1) * kTreeRows; }
PKV_HD int64_t tree_seg_cost(int rows, int pair, int nblk) {
  return kTreeSeg + (int64_t)nblk * (tree_two(rows, pair) ? kTreeTwo : kTreeOne);
}
// whole cost of a sequence (0 where it has no rows)
PKV_HD int64_t tree_seq_cost(int Hkv, int rows, int nblk) {
  const int pairs = tree_pairs(rows);
  if (pairs == 0) return 0;
  return Hkv * ((pairs - 1) * tree_seg_cost(2 * kTreeRows, 0, nblk) +
                tree_seg_cost(rows, pairs - 1, nblk));
}
// CTAs that get work, of `launched`
PKV_HD int64_t tree_shares(int64_t cost, int64_t launched) {
  const int64_t n = cost / kTreeMinShare;
  return n < 1 ? 1 : n < launched ? n : launched;
}
PKV_HD int64_t tree_share(int64_t c, int64_t cost, int64_t n) {  // first cost of share c
  return udiv64(c * cost + n - 1, n);
}

// One CTA's blocks j0 .. j0 + nblk - 1 of the `total` of a segment.
struct TreePart {
  int b, pair, h, j0, nblk, total;
  bool two;
};
// The segment at offset r of a sequence's stretch of the line, cut by `left`, the
// costs from there to the share's end.  Returns the costs from r to the segment's
// end; s.nblk may be 0.
PKV_HD int64_t tree_part(int Hkv, int rows, int nblk, int64_t r, int64_t left, TreePart& s) {
  const int pairs = tree_pairs(rows);
  const int64_t whole = Hkv * tree_seg_cost(2 * kTreeRows, 0, nblk);
  s.pair = 0;
  if (pairs > 1) {
    const int64_t at = udiv64(r, whole);
    s.pair = at < pairs - 1 ? (int)at : pairs - 1;
  }
  s.two = tree_two(rows, s.pair);
  const int w = s.two ? kTreeTwo : kTreeOne;
  const int64_t seg = tree_seg_cost(rows, s.pair, nblk);
  r -= s.pair * whole;
  s.h = (int)udiv64(r, seg);
  r -= s.h * seg;
  // block j begins at kTreeSeg + j w
  auto first = [&](int64_t x) -> int64_t {
    return x <= kTreeSeg ? 0 : udiv64(x - kTreeSeg + w - 1, w);
  };
  const int64_t j0 = first(r), j1 = first(r + left);
  s.total = nblk;
  s.j0 = (int)(j0 < nblk ? j0 : nblk);
  s.nblk = (int)(j1 < nblk ? j1 : nblk) - s.j0;
  return seg - r;
}

}  // namespace pkv
