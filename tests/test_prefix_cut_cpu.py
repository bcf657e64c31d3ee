"""How the shared prefix's work is cut into shares (pkv_prefix_line.h), walked on the
host: whatever stretch of the prefix is seen, the launched CTAs cover every unit
once, and the merge reads the slots that were written and no others."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <vector>
#include "pkv_prefix_line.h"
using namespace pkv;

// 0, or what is wrong: 1 a unit not covered, 2 covered twice, 3 a slot outside the
// workspace, 4 a slot written twice, 5 the merge reads a slot nobody wrote, 6 a
// written slot is not read.  cut: the CTAs the line is cut for (0: the launch's).
extern "C" int walk(int Hkv, int64_t rows, int64_t prefix, int sms, int seen, int64_t cut) {
  const int pairs = prefix_pairs(rows);
  const int64_t cost = prefix_cost(Hkv, prefix_blocks_of(prefix), pairs,
                                   prefix_last_weight(rows, pairs));
  const int64_t launched = prefix_ctas(cost, sms);
  if (launched < 1 || launched > sms) return 7;
  const PrefixLine line(Hkv, rows, pairs, seen, cut ? cut : launched);
  const int segs = pairs * Hkv;
  std::vector<int> unit((size_t)segs * line.nblk, 0), slot((size_t)sms + segs, 0);
  for (int64_t c = 0; c < launched && c < line.n && seen > 0; ++c) {
    int64_t x = line.share(c);
    const int64_t hi = line.share(c + 1);
    PrefixPart s;
    while (next_part(line, x, hi, s)) {
      for (int j = s.j0; j < s.j0 + s.nblk; ++j)
        if (++unit[(size_t)(s.pair * Hkv + s.h) * line.nblk + j] > 1) return 2;
      const int64_t at = line.slot(c, s.pair, s.h);
      if (at < 0 || at >= (int64_t)slot.size()) return 3;
      if (++slot[at] > 1) return 4;
    }
  }
  for (int u : unit)
    if (u != 1) return 1;
  for (int p = 0; p < pairs && seen > 0; ++p)
    for (int h = 0; h < Hkv; ++h)
      for (int64_t c = line.first_cta(p, h); c <= line.last_cta(p, h); ++c) {
        const int64_t at = line.slot(c, p, h);
        if (at < 0 || at >= (int64_t)slot.size() || slot[at] != 1) return 5;
        slot[at] = 2;
      }
  for (int s : slot)
    if (s == 1) return 6;
  return 0;
}

// every stretch of a prefix from nothing to all of it; the first that goes wrong
extern "C" int64_t sweep(int Hkv, int64_t rows, int64_t prefix, int sms) {
  for (int64_t seen = 0; seen <= prefix; seen += seen + 128 <= prefix ? 128 : 1) {
    const int e = walk(Hkv, rows, prefix, sms, (int)seen, 0);
    if (e) return seen * 10 + e;
  }
  return -1;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("cut")
    (d / "cut.cpp").write_text(SOURCE)
    so = str(d / "cut.so")
    csrc = os.path.join(ROOT, "paged_kv_cache_250_gb300", "csrc")
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I", csrc,
                    str(d / "cut.cpp"), "-o", so], check=True)
    x = ctypes.CDLL(so)
    i, l = ctypes.c_int, ctypes.c_int64
    x.walk.argtypes, x.walk.restype = [i, l, l, i, i, l], i
    x.sweep.argtypes, x.sweep.restype = [i, l, l, i], l
    return x


@pytest.mark.parametrize("sms", [152, 148, 13, 1])
@pytest.mark.parametrize("Hkv", [1, 2, 3, 8, 32])
@pytest.mark.parametrize("rows", [4, 48, 128, 129, 256, 257, 400, 1024, 24000])
def test_every_stretch_is_covered_once(lib, sms, Hkv, rows):
    for blocks in (1, 2, 17, 19, 20, 39, 40, 58, 77, 115, 153, 256):
        if rows == 24000 and blocks > 40:
            continue
        for tokens in (128 * blocks, 128 * blocks - 112):
            assert lib.sweep(Hkv, rows, tokens, sms) == -1, (blocks, tokens)


def test_the_sizes_at_which_the_count_of_ctas_falls(lib):
    """64 sequences of 4 heads per KV head behind 2560 tokens, none longer than
    2432; one tile of rows behind 5120, none longer than 4864."""
    assert lib.walk(8, 256, 2560, 152, 2432, 0) == 0
    assert lib.walk(8, 128, 5120, 152, 4864, 0) == 0


def test_a_cut_for_more_ctas_than_were_launched_shows(lib):
    assert lib.walk(8, 256, 2560, 152, 2432, 152) == 1
    assert lib.walk(8, 128, 5120, 152, 4864, 152) == 1
