"""How decode attention behind a shared prefix divides its work, on the CPU: every tile and
block in one share, every share's part in a slot of its own, the join's account the same as the
CTAs'."""
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
#include "ee_shared_plan.cuh"
using namespace ee;

#define CHECK(...) do { if (!(__VA_ARGS__)) return __LINE__; } while (0)

// 0, or the line of the first check that fails.  n: tokens of each sequence.
template <int G>
int divide(int hkv, int batch, int prefix, int hd, int ctas, const int* n, int* n_pre) {
  Pieces<G> p;
  int longest = 0, pairs = 0, base[64];
  for (int s = 0; s < batch; ++s) longest = n[s] > longest ? n[s] : longest;
  p.init(hkv, batch, prefix, longest >= prefix);
  p.own_end = 0;
  for (int s = 0; s < batch; ++s) {
    base[s] = p.own_end;
    p.own_end += hkv * p.own_places(n[s]);
    pairs += p.own_places(n[s]) > 0 ? hkv : 0;
  }
  uint32_t best = ~0u;
  for (int i = 0; i < 32; ++i) {
    const uint32_t e = p.estimate(i, ctas, pairs, hd);
    best = e < best ? e : best;
  }
  p.share_out(ctas, (int)(best & 255));
  *n_pre = p.n_pre;
  CHECK(p.n_pre >= 0 && p.n_pre <= ctas);
  if (p.pre_end > 0) CHECK(p.n_pre >= 1);
  if (p.own_end > 0) CHECK(p.n_pre < ctas);

  const int64_t pre_slots = prefix_slots(batch, G, hkv, prefix);
  std::set<int64_t> slots;
  std::map<std::pair<int, int>, std::set<int>> pieces;  // of a unit (row tile, head)
  std::map<std::pair<int, int>, std::vector<int>> seen;
  int total = 0;
  for (int me = 0; me < p.n_pre; ++me) {
    int c = me * p.each_pre, kind = 2;
    for (;;) {
      const Work w = p.prefix_at(&c, me);
      if (!w.kind) break;
      const int rt = w.s * G / 256;
      CHECK(w.s * G % 256 == 0 && w.rows == p.rows_of(rt) && w.kind == (w.rows > 128 ? 2 : 1));
      CHECK(w.kind <= kind);  // wide units first
      kind = w.kind;
      CHECK(w.tiles > 0 && w.first % 8 == 0 && w.first / 8 + w.tiles <= p.tiles());
      CHECK(w.have > (w.tiles - 1) * kKeys && w.have <= w.tiles * kKeys && w.first * 16 + w.have <= p.pre * 16);
      CHECK(w.have % kKeys == 0 || w.first * 16 + w.have == p.pre * 16);
      CHECK(w.slot == p.pre_slot(rt, w.g, me) && w.slot >= 0 && w.slot < pre_slots && slots.insert(w.slot).second);
      auto& tiles = seen[{rt, w.g}];
      CHECK((int)tiles.size() == w.first / 8);  // one after the other
      for (int k = 0; k < w.tiles; ++k) tiles.push_back(me);
      pieces[{rt, w.g}].insert(me);
      total += w.tiles;
    }
  }
  int units = 0;
  for (int rt = 0; rt < 2 && p.pre > 0; ++rt) {
    if (p.rows_of(rt) <= 0) continue;
    for (int g = 0; g < hkv; ++g, ++units) {
      CHECK((int)seen[{rt, g}].size() == p.tiles());
      const auto r = p.prefix_range(rt, g);
      CHECK(r.first >= 0 && r.first <= r.last && r.last < p.n_pre && r.last - r.first + 1 <= kMaxPieces);
      for (int i = 0; i < p.n_pre; ++i)
        CHECK((i >= r.first && i <= r.last && r.has(i)) == (pieces[{rt, g}].count(i) == 1));
    }
  }
  CHECK(total == units * p.tiles());
  CHECK(units == 0 || p.rows_of(0) > 128 || p.rows_of(1) <= 0);

  slots.clear();
  pieces.clear();
  std::map<std::pair<int, int>, int> blocks;
  const int streams = 2 * (ctas - p.n_pre);
  CHECK(p.own_end == 0 || (int64_t)streams * p.each_own >= p.own_end);
  for (int me = 0, s = 0; me < streams; ++me) {
    int c = me * p.each_own;
    const int stop = (me + 1) * p.each_own < p.own_end ? (me + 1) * p.each_own : p.own_end;
    for (s = 0; c < stop;) {
      while (c >= base[s] + hkv * p.own_places(n[s])) ++s;
      Own w;
      const int before = c;
      const bool any = p.own_at(&c, me, s, base[s], n[s], &w);
      CHECK(c > before && w.g >= 0 && w.g < hkv);
      if (!any) continue;
      CHECK(w.blocks > 0 && w.first == p.first_own(n[s]) + blocks[{s, w.g}]);
      CHECK(w.row == (prefix > 0 && p.first_own(n[s]) == 0 ? 0 : s));
      CHECK(w.have > (w.blocks - 1) * 16 && w.have <= w.blocks * 16 && w.first * 16 + w.have <= n[s]);
      CHECK(w.slot == p.own_slot(s, w.g, me) && w.slot >= 0 && w.slot < own_slots(batch, hkv) && slots.insert(w.slot).second);
      blocks[{s, w.g}] += w.blocks;
      pieces[{s, w.g}].insert(me);
    }
  }
  for (int s = 0; s < batch; ++s)
    for (int g = 0; g < hkv; ++g) {
      CHECK((blocks[{s, g}]) == p.own_blocks(n[s]));
      if (p.own_blocks(n[s]) == 0) continue;
      const auto r = p.own_range(base[s], g, n[s]);
      CHECK(r.first >= 0 && r.first <= r.last && r.last < streams);
      const auto& has = pieces[{s, g}];
      CHECK(*has.begin() >= r.first && *has.rbegin() <= r.last);
      for (int i = r.first; i <= r.last; ++i) CHECK(r.has(i) == (has.count(i) == 1));
    }
  return 0;
}

extern "C" int check(int G, int hkv, int batch, int prefix, int hd, int ctas, const int* n, int* n_pre) {
  if (G == 1) return divide<1>(hkv, batch, prefix, hd, ctas, n, n_pre);
  if (G == 2) return divide<2>(hkv, batch, prefix, hd, ctas, n, n_pre);
  if (G == 4) return divide<4>(hkv, batch, prefix, hd, ctas, n, n_pre);
  return divide<8>(hkv, batch, prefix, hd, ctas, n, n_pre);
}
"""


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, out = d / "plan.cpp", d / "plan.so"
    src.write_text(SOURCE)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-ftrapv", "-I" + build.CSRC, "-shared", "-fPIC", str(src), "-o", str(out)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(str(out))

    def run(G, hkv, prefix, ctxs, ctas, hd=128):
        n, n_pre = np.array(ctxs, np.int32), ctypes.c_int(0)
        line = lib.check(G, hkv, len(n), prefix, hd, ctas, ctypes.c_void_p(n.ctypes.data), ctypes.byref(n_pre))
        assert line == 0, (f"line {line}: {SOURCE.splitlines()[line - 1].strip()}", G, hkv, prefix, list(ctxs), ctas)
        return n_pre.value

    return run


@pytest.mark.parametrize("G,hkv,prefix,ctxs", [
    (4, 8, 512, [513, 600, 530, 1100]), (8, 8, 14992, [15000 + 20 * i for i in range(64)]), (4, 8, 2048, [2048 + 9 * i for i in range(32)]),
    (8, 1, 16, [16, 17, 0, 5]), (1, 1, 0, [1]), (2, 2, 320, [100, 50, 319]), (8, 2, 320, [0, 400, 16, 1]), (4, 3, 0, [16384] * 64),
    (8, 8, 16384, [16384] * 64), (8, 1024, 16384, [16384] * 64), (1, 1024, 16, [40] * 64), (4, 8, 256, [0] * 32),
])
def test_shapes(check, G, hkv, prefix, ctxs):
    for ctas in (2, 3, 31, 33, 132, 148, 152, 160):
        for hd in (64, 128):
            n_pre = check(G, hkv, prefix, ctxs, ctas, hd)
            whole = prefix >= 16 and max(ctxs) >= prefix
            assert (n_pre > 0) == whole


def test_a_single_cta(check):
    """Work of one kind takes every CTA, also where there is one."""
    assert check(1, 1, 0, [40], 1) == 0
    assert check(4, 1, 16, [16], 1) == 1


def test_drawn(check):
    r = np.random.default_rng(5)
    kinds = set()
    for _ in range(1500):
        batch = int(np.exp(r.uniform(0, np.log(64.99))))
        prefix = int(np.exp(r.uniform(0, np.log(16384)))) // 16 * 16
        most = int(np.exp(r.uniform(0, np.log(16384))))
        ctxs = np.minimum(16384, r.integers(0, most + 1, batch) + (prefix if r.random() < 0.8 else 0))
        ctxs[r.random(batch) < r.choice([0, 0.1])] = 0
        if r.random() < 0.2:
            ctxs[r.integers(batch)] = prefix // 2
        G, hkv, ctas = int(r.choice([1, 2, 4, 8])), int(r.choice([1, 2, 3, 8, 16])), int(r.integers(2, 161))
        n_pre = check(G, hkv, prefix, ctxs, ctas, int(r.choice([64, 128])))
        kinds.add((n_pre == 0, n_pre == ctas))
    assert len(kinds) == 3   # own blocks alone, the prefix alone, both
