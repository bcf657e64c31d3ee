"""How the tree kernel's work is cut into shares, walked on the host with the
kernel's own header: every block of every segment belongs to one CTA, and the
merge finds the parts of every segment that a share boundary cuts."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_cache_250_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <tuple>
#include <vector>
#include "pkv_tree_line.h"
using namespace pkv;

static int fail(const char* what, long a, long b) {
  std::printf("%s %ld %ld\n", what, a, b);
  return 1;
}

// One line of the work (two: segments of two tiles).
static int walk(bool two, const std::vector<int>& rows, const std::vector<int>& ctx, int Hkv,
                int most) {
  const int B = (int)rows.size();
  std::vector<int64_t> line(B + 1, 0);
  for (int b = 0; b < B; ++b)
    line[b + 1] = line[b] + tree_seq_cost(two, Hkv, rows[b], tree_blocks(ctx[b]));
  const int64_t cost = line[B], n = tree_shares(cost, most);
  if (n < 1 || n > most) return fail("shares", n, most);
  std::map<std::tuple<int, int, int>, std::vector<int>> seen;   // segment -> shares of its blocks
  struct Left { int parts = 0; std::tuple<int, int, int> seg; };  // where a segment starts
  std::vector<Left> left(most);
  std::vector<std::tuple<int, int, int>> head(most, {-1, -1, -1});
  int64_t longest = 0;
  for (int64_t c = 0; c < n; ++c) {
    int64_t at = cost ? tree_share(c, cost, n) : 0;
    const int64_t hi = cost ? tree_share(c + 1, cost, n) : 0;
    if (c == 0 && at != 0) return fail("start", at, 0);
    if (c == n - 1 && hi != cost) return fail("end", hi, cost);
    longest = std::max(longest, hi - at);
    int parts = 0, b = 0;
    while (at < hi) {
      while (line[b + 1] <= at) ++b;
      TreePart s;
      s.b = b;
      const int64_t step = tree_part(two, rows[b], tree_blocks(ctx[b]), at - line[b], hi - at, s);
      if (step <= 0) return fail("step", step, at);
      at += step;
      if (s.nblk <= 0) continue;
      if (s.h < 0 || s.h >= Hkv || s.row0 < 0 || s.row0 >= rows[b] || s.row0 % 256)
        return fail("segment", s.row0, s.h);
      if ((rows[b] - s.row0 > 128) != two) return fail("tiles", rows[b], s.row0);
      const auto key = std::make_tuple(b, s.row0, s.h);
      auto& v = seen[key];
      for (int j = 0; j < s.nblk; ++j) {
        if ((int)v.size() != s.j0 + j) return fail("order", v.size(), s.j0 + j);
        v.push_back((int)c);
      }
      const bool ends = s.j0 + s.nblk == s.total;
      if (s.j0 > 0) {
        if (parts != 0) return fail("not the first part", c, parts);
        head[c] = key;
      } else if (!ends) {
        if (left[c].parts) return fail("two that go on", c, parts);
        left[c].parts = (int)(tree_share_of(at - kTreeBlock, cost, n) - c) + 1;
        left[c].seg = key;
      }
      ++parts;
    }
  }
  if (longest > (cost + n - 1) / n) return fail("longest", longest, cost / n);
  size_t segs = 0;
  for (int b = 0; b < B; ++b) segs += (size_t)Hkv * tree_segs(two, rows[b]);
  if (seen.size() != segs) return fail("segments", seen.size(), segs);
  int cut = 0;
  for (auto& kv : seen) {
    if ((int)kv.second.size() != tree_blocks(ctx[std::get<0>(kv.first)]))
      return fail("blocks", std::get<0>(kv.first), std::get<1>(kv.first));
    cut += kv.second.front() != kv.second.back();
  }
  for (int c = 0; c < most; ++c) {
    if (!left[c].parts) continue;
    --cut;
    for (int k = c + 1; k < c + left[c].parts; ++k)
      if (k >= most || head[k] != left[c].seg) return fail("part", c, k);
    if (left[c].parts < 2 || seen[left[c].seg].back() != c + left[c].parts - 1)
      return fail("last", c, left[c].parts);
  }
  if (cut != 0) return fail("cut segments", cut, 0);
  return 0;
}

// Both lines, for `ctas` CTAs; every row in one segment.
static int both(const std::vector<int>& rows, const std::vector<int>& ctx, int Hkv, int ctas) {
  for (size_t b = 0; b < rows.size(); ++b) {
    int next = 0;
    for (int s = 0; s < tree_segs(true, rows[b]); ++s) {
      if (tree_row0(true, rows[b], s) != next) return fail("rows of line 2", b, s);
      next += 256;
    }
    if (tree_segs(false, rows[b])) {
      if (tree_row0(false, rows[b], 0) != next) return fail("rows of line 1", b, next);
      next += 128;
    }
    if (next < rows[b] || (rows[b] == 0 && next)) return fail("rows", rows[b], next);
  }
  const int r = walk(true, rows, ctx, Hkv, ctas);
  return r ? r : walk(false, rows, ctx, Hkv, 2 * ctas);
}

int main() {
  std::mt19937 g(5);
  auto draw = [&](int lo, int hi) { return lo + (int)(g() % (uint32_t)(hi - lo + 1)); };
  for (int it = 0; it < 4000; ++it) {
    const int B = draw(1, it % 3 == 0 ? 300 : 12), G = 1 << draw(0, 3), Hkv = draw(1, 8);
    const int launched = it % 4 == 0 ? draw(1, 200) : 152;
    const int most = it % 5 == 0 ? 40000 : it % 5 == 1 ? 300 : 4000;
    std::vector<int> rows, ctx;
    for (int b = 0; b < B; ++b) {
      const int n = draw(0, 9) == 0 ? 0 : draw(1, 64);
      rows.push_back(n * G);
      ctx.push_back(n + draw(0, most));
    }
    if (int r = both(rows, ctx, Hkv, launched)) { std::printf("iteration %d\n", it); return r; }
  }
  if (both({0, 0}, {5, 0}, 2, 152)) return 1;
  if (both({512}, {2147483647}, 1, 152)) return 1;
  if (both({512, 8, 0, 136}, {64, 1, 0, 2147483000}, 1, 152)) return 1;
  const int64_t far = ((int64_t)1 << 32) - 1;  // the largest cost a call may have
  if (tree_share(152, far, 152) != far || tree_shares(far, 152) != 152 ||
      tree_share_of(far - 1, far, 304) != 303)
    return 1;
  std::puts("ok");
  return 0;
}
"""


def test_every_block_once_and_every_cut_segment_merged(tmp_path):
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


if __name__ == "__main__":
    pytest.main([__file__])
