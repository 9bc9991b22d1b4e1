"""How decode attention over the eight-bit cache cuts its blocks into pieces, on the CPU: every
block in one share, parts in slots of their own, the join's account the same as the CTAs'."""
import ctypes
import subprocess

import numpy as np
import pytest

from early_exit_decoding_layer_gb300 import build

SOURCE = """
#include <cstdint>
#include <map>
#include <set>
#include <vector>
#include "ee_decode_pieces.cuh"
using namespace ee;

#define CHECK(...) do { if (!(__VA_ARGS__)) return __LINE__; } while (0)

// 0, or the line of the first check that fails.  n: tokens of each sequence; whole: a CTA takes the pairs that
// begin in its piece.  start: whether beginnings count.
extern "C" int check(int hkv, int batch, int ctas, int least, int whole, const int* n, int* start) {
  DecodePieces p;
  int blocks = 0, pairs = 0, total = 0, base[64];
  for (int s = 0; s < batch; ++s) {
    blocks += (n[s] + 15) / 16;
    pairs += n[s] > 0;
  }
  p.cut(hkv, blocks, pairs, ctas, least);
  for (int c = 8; c <= 32 && !whole; c += 8) {
    int parts = 0;
    for (int s = 0; s < batch; ++s) parts += ((n[s] + 15) / 16 + c - 1) / c;
    p.cut_alone(c, parts, ctas);
  }
  *start = p.start;
  for (int s = 0; s < batch; ++s) {
    base[s] = total;
    total += hkv * p.places((n[s] + 15) / 16);
  }
  CHECK((int64_t)ctas * p.each >= total && p.each >= 8);
  auto next_pair = [&](int c) {
    for (int s = 0; s < batch; ++s)
      for (int g = 0, len = p.places((n[s] + 15) / 16); g < hkv && len > 0; ++g)
        if (base[s] + g * len >= c) return base[s] + g * len;
    return total;
  };
  std::map<std::pair<int, int>, int> seen;
  std::map<std::pair<int, int>, std::vector<int>> slots;  // of a pair, in the CTAs' order
  std::set<int> taken;
  for (int me = 0; me < ctas; ++me) {
    int begin = total < me * p.each ? total : me * p.each, end = total < begin + p.each ? total : begin + p.each;
    if (whole) {
      begin = next_pair(begin);
      end = next_pair(end);
    }
    int parts = 0;
    for (int c = begin, s = 0; c < end;) {
      while (c >= base[s] + hkv * p.places((n[s] + 15) / 16)) ++s;
      Share w;
      const int before = c;
      const bool any = p.share(&c, me, begin, end, s, base[s], n[s], &w);
      CHECK(c > before);
      if (!any) continue;
      const int nb = (n[s] + 15) / 16;
      CHECK(w.s == s && w.g >= 0 && w.g < hkv && w.blocks > 0 && w.blocks <= nb);
      CHECK(w.first == (seen[{s, w.g}]));
      CHECK(w.have > (w.blocks - 1) * 16 && w.have <= w.blocks * 16 && w.first * 16 + w.have <= n[s]);
      CHECK((w.slot < 0) == (w.blocks == nb));
      CHECK(!whole || w.slot < 0);
      seen[{s, w.g}] += w.blocks;
      if (w.slot >= 0) {
        CHECK(w.slot / 2 == me && taken.insert(w.slot).second && ++parts <= 2);
        slots[{s, w.g}].push_back(w.slot);
      }
    }
  }
  for (int s = 0; s < batch; ++s)
    for (int g = 0; g < hkv; ++g) {
      const int nb = (n[s] + 15) / 16;
      CHECK((seen[{s, g}]) == nb);
      if (whole) continue;  // no join
      const auto r = p.parts(base[s] + g * p.places(nb), nb);
      const auto& written = slots[{s, g}];
      CHECK(nb > 0 ? r.count >= 1 : r.count == 0);
      CHECK((r.count < 2) == written.empty());
      if (r.count < 2) continue;
      CHECK((int)written.size() == r.count);
      for (int k = 0; k < r.count; ++k) CHECK(written[k] == r.slot(k));
    }
  return 0;
}
"""


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    d = tmp_path_factory.mktemp("pieces")
    src, out = d / "pieces.cpp", d / "pieces.so"
    src.write_text(SOURCE)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-ftrapv", "-I" + build.CSRC, "-shared", "-fPIC", str(src), "-o", str(out)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(str(out))

    def run(hkv, ctxs, ctas, whole=False, least=8):
        n, start = np.array(ctxs, np.int32), ctypes.c_int(0)
        line = lib.check(hkv, len(n), ctas, least, int(whole), ctypes.c_void_p(n.ctypes.data), ctypes.byref(start))
        assert line == 0, (f"line {line}: {SOURCE.splitlines()[line - 1].strip()}", hkv, list(ctxs), ctas)
        return start.value

    return run


@pytest.mark.parametrize("hkv,ctxs", [
    (8, [2113]), (8, [16384] * 16), (2, [33]), (1, [1]), (8, [0, 1, 0, 16, 17, 0]), (8, [0] * 5), (1024, [16384] * 64), (1024, [39] * 64),
    (8, [500] * 8), (8, [300] * 64), (1, [16384]), (3, [16384, 0, 1, 5000, 129]),
])
def test_shapes(check, hkv, ctxs):
    for ctas in (1, 2, 31, 148, 296, 304, 444, 456, 480):
        check(hkv, ctxs, ctas)
        if max(ctxs) <= 128:
            check(hkv, ctxs, ctas, whole=True)


def test_drawn(check):
    r = np.random.default_rng(6)
    starts = set()
    for _ in range(1500):
        batch = int(np.exp(r.uniform(0, np.log(64.99))))
        ctxs = r.integers(0, int(np.exp(r.uniform(0, np.log(16384)))) + 1, batch)
        ctxs[r.random(batch) < r.choice([0, 0.2])] = 0
        hkv, ctas = int(r.choice([1, 2, 3, 8, 16])), int(r.integers(1, 481))
        starts.add(check(hkv, ctxs, ctas))
        check(hkv, np.minimum(ctxs, 128), ctas, whole=True)
    assert starts == {0, 6}   # beginnings that count, and pairs cut by themselves
