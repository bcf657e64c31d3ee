// pkv_tree_line.h -- how the tree kernel's work is cut into shares.  Needs no CUDA.
//
// The rows of a (sequence, KV head), its nodes times the g query heads of the KV
// head, are cut into pairs of 128-row tiles, and what is left beyond whole pairs
// into one more: a pair whose second tile holds rows is a segment of line 2, the
// last one without a segment of line 1.  A segment's units are the blocks of 128
// cached tokens.  Each line holds its segments sequence by sequence, head by
// head, pair by pair, where a segment's start costs kTreeSeg and a block
// kTreeBlock, and is cut into equal shares; a unit belongs to the share that its
// first cost lies in.
#pragma once

#include "pkv_hd.h"

namespace pkv {

constexpr int kTreeRows = 128, kTreeTok = 128;  // rows of a tile, tokens of a block
constexpr int kTreeBlock = 2, kTreeSeg = 4;
constexpr int kTreeMinShare = 2;  // a share is worth at least a block (10.7 us for one
                                  // sequence of 708 tokens, 12.6 for two blocks)
constexpr int kTreeMaxBatch = 3328, kTreeMaxCtas = 256;
static_assert(kTreeMinShare >= kTreeBlock, "no share without a block inside a segment");

PKV_HD int tree_blocks(int ctx) { return (int)(((int64_t)ctx + kTreeTok - 1) / kTreeTok); }
// segments of a (sequence, KV head) on line 2 (two) or 1, and the first row of one
PKV_HD int tree_segs(bool two, int rows) {
  const int pairs = (rows + kTreeRows - 1) / (2 * kTreeRows);  // with two tiles
  return two ? pairs : rows > 2 * kTreeRows * pairs ? 1 : 0;
}
PKV_HD int tree_row0(bool two, int rows, int seg) {
  return 2 * kTreeRows * (two ? seg : tree_segs(true, rows));
}
// (Costs along a line are 32-bit: a call whose line could be longer is refused.)
PKV_HD uint32_t tree_seg_cost(int nblk) { return kTreeSeg + (uint32_t)nblk * kTreeBlock; }
// whole cost of a sequence on a line
PKV_HD int64_t tree_seq_cost(bool two, int Hkv, int rows, int nblk) {
  return (int64_t)Hkv * tree_segs(two, rows) * tree_seg_cost(nblk);
}
// Shares that get work, of at most `most`.
PKV_HD int64_t tree_shares(int64_t cost, int64_t most) {
  const int64_t n = cost / kTreeMinShare;
  return n < 1 ? 1 : n < most ? n : most;
}
PKV_HD int64_t tree_share(int64_t c, int64_t cost, int64_t n) {  // first cost of share c
  return udiv64(c * cost + n - 1, n);
}
PKV_HD int64_t tree_share_of(int64_t x, int64_t cost, int64_t n) {  // the share that x lies in
  return udiv64(x * n, cost);
}

// A share's blocks j0 .. j0 + nblk - 1 of the `total` of a segment.
struct TreePart {
  int b, h, row0, j0, nblk, total;
};
// The segment at offset r of a sequence's stretch of a line, cut by `left`, the
// costs from there to the share's end.  Returns the costs from r to the segment's
// end; s.nblk may be 0.
PKV_HD uint32_t tree_part(bool two, int rows, int nblk, uint32_t r, uint32_t left, TreePart& s) {
  const uint32_t seg = tree_seg_cost(nblk);
  const int per = tree_segs(two, rows);
  const int at = (int)(r / seg);
  r -= (uint32_t)at * seg;
  s.h = per == 1 ? at : at / per;
  s.row0 = tree_row0(two, rows, at - s.h * per);
  // block j begins at kTreeSeg + j kTreeBlock
  auto first = [&](uint32_t x) -> int {
    if (x >= seg) return nblk;
    return x <= kTreeSeg ? 0 : (int)((x - kTreeSeg + kTreeBlock - 1) / kTreeBlock);
  };
  s.total = nblk;
  s.j0 = first(r);
  s.nblk = first(left < seg - r ? r + left : seg) - s.j0;
  return seg - r;
}

}  // namespace pkv
