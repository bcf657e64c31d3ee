// pkv_prefix_line.h -- how the prefix kernel's work is cut into shares, and which
// parts of it the merge finds.  Needs no CUDA.
//
// The units (pair of 128-row tiles, KV head, block of 128 tokens) lie on one line:
// pair-major, then KV head, then block.  A block of a pair costs w = 2, or 1 where
// the second tile is empty (only in the last pair; two such blocks run side by
// side).  The line holds the blocks that some sequence sees; it is cut into n
// equal shares, one per CTA.
#pragma once

#include "pkv_hd.h"

namespace pkv {

constexpr int kPrefixRows = 128, kPrefixTok = 128;  // rows of a tile, tokens of a block

PKV_HD int64_t prefix_blocks_of(int64_t tokens) {
  return (tokens + kPrefixTok - 1) / kPrefixTok;
}
PKV_HD int32_t prefix_pairs(int64_t rows) {  // rows: those of a KV head
  return (int32_t)((rows + 2 * kPrefixRows - 1) / (2 * kPrefixRows));
}
PKV_HD int prefix_last_weight(int64_t rows, int32_t pairs) {
  return (2 * (int64_t)pairs - 1) * kPrefixRows < rows ? 2 : 1;
}
PKV_HD int64_t prefix_cost(int32_t Hkv, int64_t blocks, int32_t pairs, int last_weight) {
  return (int64_t)Hkv * blocks * (2 * (pairs - 1) + last_weight);
}

// CTAs to launch for a prefix of the given whole cost on `sms` SMs.  In units of
// cost 2 the longest share is m = ceil(units / sms); up to m = 4, as many CTAs as
// shares of m take, no more: fewer partials in the same time.  64 sequences with own
// parts of up to 512 tokens, 32/8 heads of 128, 152 SMs, a call with that many CTAs
// and with one per SM, in us:
//   m  prefix  CTAs                 m  prefix  CTAs
//   2    2560    80  31.0 / 37.1    4    7424   116  38.9 / 41.7
//   2    3584   112  34.8 / 37.8    4    8192   128  40.2 / 42.3
//   3    4992   104  35.9 / 39.6    5    9856   124  41.7 / 43.9
//   3    6144   128  38.3 / 40.5    8   16384   128  49.5 / 49.7
// (m = 5 to 7 would gain 2.2, 1.8 and 1.4 us too; the limit has not followed.)  The
// count falls where m steps up, so it belongs to the launch alone: a cut of less than
// the whole prefix (see PrefixLine) goes by the CTAs that were launched.
PKV_HD int64_t prefix_ctas(int64_t cost, int32_t sms) {
  const int64_t units = cost >> 1 > 0 ? cost >> 1 : 1;
  for (int m = 1; m <= 4; ++m)
    if (units <= (int64_t)m * sms) return ((uint32_t)units + m - 1) / m;
  return sms;
}

struct PrefixLine {
  int Hkv, pairs, nblk, last_w;
  int64_t cost, n;  // whole cost; CTAs with work
  // `rows` query rows per KV head, `seen` tokens of the prefix, `launched` CTAs.
  // A share is at least one unit, so every CTA between a segment's first and last
  // has a part of it.
  PKV_HD PrefixLine(int32_t Hkv_, int64_t rows, int32_t pairs_, int seen, int64_t launched)
      : Hkv(Hkv_), pairs(pairs_), nblk((int)prefix_blocks_of(seen)),
        last_w(prefix_last_weight(rows, pairs_)) {
    cost = prefix_cost(Hkv, nblk, pairs, last_w);
    const int64_t units = cost >> 1 > 0 ? cost >> 1 : 1;
    n = launched < units ? launched : units;
  }
  PKV_HD int weight(int pair) const { return pair == pairs - 1 ? last_w : 2; }
  PKV_HD int64_t start(int pair, int h) const {
    return (int64_t)Hkv * nblk * 2 * pair + (int64_t)h * nblk * weight(pair);
  }
  // first cost of CTA c
  PKV_HD int64_t share(int64_t c) const { return udiv64(c * cost + n - 1, n); }
  PKV_HD int64_t cta_of(int64_t x) const { return udiv64(x * n, cost); }
  // first and last CTA with a part of a segment (pair, KV head)
  PKV_HD int64_t first_cta(int pair, int h) const { return cta_of(start(pair, h)); }
  PKV_HD int64_t last_cta(int pair, int h) const {
    return cta_of(start(pair, h) + (int64_t)(nblk - 1) * weight(pair));
  }
  // CTA c leaves its part of a segment in slot c + segment: two streams of 128 rows
  PKV_HD int64_t slot(int64_t c, int pair, int h) const {
    return c + (int64_t)pair * Hkv + h;
  }
};

// One CTA's blocks of one segment.
struct PrefixPart {
  int pair, h, j0, nblk;
  bool two;
};
// Steps through the segments that the costs [x, hi) cross; false at the end.
// A unit belongs to the share its first cost lies in.
PKV_HD bool next_part(const PrefixLine& ln, int64_t& x, int64_t hi, PrefixPart& s) {
  while (x < hi) {
    const int64_t per = (int64_t)ln.Hkv * ln.nblk * 2;
    s.pair = 0;
    if (ln.pairs > 1) {
      const int64_t at = udiv64(x, per);
      s.pair = at < ln.pairs - 1 ? (int)at : ln.pairs - 1;
    }
    const int w = ln.weight(s.pair);
    s.two = w == 2;
    const int64_t seg = (int64_t)ln.nblk * w;
    s.h = (int)udiv64(x - per * s.pair, seg);
    const int64_t s0 = ln.start(s.pair, s.h);
    s.j0 = (int)((x - s0 + w - 1) >> (w - 1));  // w is 1 or 2
    const int64_t j1 = (hi - s0 + w - 1) >> (w - 1);
    s.nblk = (int)((j1 < ln.nblk ? j1 : ln.nblk) - s.j0);
    x = s0 + seg;
    if (s.nblk > 0) return true;
  }
  return false;
}

}  // namespace pkv
