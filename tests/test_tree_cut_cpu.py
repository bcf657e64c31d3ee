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

static int walk(const std::vector<int>& rows, const std::vector<int>& ctx, int Hkv, int launched) {
  const int B = (int)rows.size();
  std::vector<int64_t> pfx(B + 1, 0);
  for (int b = 0; b < B; ++b)
    pfx[b + 1] = pfx[b] + tree_seq_cost(Hkv, rows[b], tree_blocks(ctx[b]));
  const int64_t cost = pfx[B], n = tree_shares(cost, launched);
  if (n < 1 || n > launched) return fail("shares", n, launched);
  std::map<std::tuple<int, int, int>, std::vector<int>> seen;   // segment -> blocks, in order
  struct Meta { bool tail = false, head = false, head_ends = false; std::tuple<int, int, int> seg, head_seg; };
  std::vector<Meta> meta(launched);
  int64_t longest = 0;
  for (int64_t c = 0; c < n; ++c) {
    int64_t at = tree_share(c, cost, n);
    const int64_t hi = tree_share(c + 1, cost, n);
    if (c == 0 && at != 0) return fail("start", at, 0);
    if (c == n - 1 && hi != cost) return fail("end", hi, cost);
    int parts = 0;
    while (at < hi) {
      int a = 0, z = B;
      while (z - a > 1) {
        const int mid = (a + z) >> 1;
        if (pfx[mid] <= at) a = mid; else z = mid;
      }
      if (rows[a] == 0) return fail("empty sequence", a, at);
      TreePart s;
      s.b = a;
      const int64_t step = tree_part(Hkv, rows[a], tree_blocks(ctx[a]), at - pfx[a], hi - at, s);
      if (step <= 0) return fail("step", step, at);
      at += step;
      if (s.nblk <= 0) continue;
      if (s.pair >= tree_pairs(rows[a]) || s.h >= Hkv || s.pair < 0 || s.h < 0)
        return fail("segment", s.pair, s.h);
      if (s.two != tree_two(rows[a], s.pair)) return fail("two", a, s.pair);
      const auto key = std::make_tuple(a, s.pair, s.h);
      auto& v = seen[key];
      for (int j = 0; j < s.nblk; ++j) {
        if ((int)v.size() != s.j0 + j) return fail("order", v.size(), s.j0 + j);
        v.push_back((int)c);
      }
      const bool head = s.j0 > 0, ends = s.j0 + s.nblk == s.total;
      if (head) {
        if (parts != 0) return fail("head is not the first part", c, parts);
        meta[c].head = true;
        meta[c].head_ends = ends;
        meta[c].head_seg = key;
      } else if (!ends) {
        if (meta[c].tail) return fail("two tails", c, parts);
        meta[c].tail = true;
        meta[c].seg = key;
      }
      ++parts;
    }
    longest = std::max(longest, hi - tree_share(c, cost, n));
  }
  if (longest > (cost + n - 1) / n) return fail("longest", longest, cost / n);
  for (int b = 0; b < B; ++b)
    for (int pr = 0; pr < tree_pairs(rows[b]); ++pr)
      for (int h = 0; h < Hkv; ++h) {
        auto it = seen.find(std::make_tuple(b, pr, h));
        if (it == seen.end() || (int)it->second.size() != tree_blocks(ctx[b]))
          return fail("blocks", b, pr);
      }
  int cut = 0;
  for (auto& kv : seen) cut += kv.second.front() != kv.second.back();
  for (int c = 0; c < launched; ++c) {
    if (!meta[c].tail) continue;
    --cut;
    int last = c + 1;
    while (last < launched - 1 && !meta[last].head_ends) ++last;
    for (int k = c + 1; k <= last; ++k)
      if (k >= launched || !meta[k].head || meta[k].head_seg != meta[c].seg)
        return fail("part", c, k);
    if (!meta[last].head_ends || seen[meta[c].seg].back() != last) return fail("last", c, last);
  }
  if (cut != 0) return fail("cut segments", cut, 0);
  return 0;
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
    if (int r = walk(rows, ctx, Hkv, launched)) { std::printf("iteration %d\n", it); return r; }
  }
  if (walk({0, 0}, {5, 0}, 2, 152)) return 1;
  if (walk({512}, {2147483647}, 8, 152)) return 1;
  std::vector<int> many(4000, 512), far(4000, 8000000);
  if (walk({512, 8, 0, 136}, {64, 1, 0, 2147483000}, 1, 152)) return 1;
  int64_t c = 0;
  for (int b = 0; b < 4000; ++b) c += tree_seq_cost(8, many[b], tree_blocks(far[b]));
  if (tree_share(152, c, 152) != c || tree_shares(c, 152) != 152) return 1;
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
