"""Host logic of the scored decode's batches: the split length chosen from the
lengths, and the splits launched for.  Compiled as plain C++ against
csrc/kvq_batch_splits.h, no GPU involved."""
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "quantized_kv_cache_append_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "kvq_batch_splits.h"
int main() {
  char what;
  while (scanf(" %c", &what) == 1) {
    if (what == 'i') {
      long long cap; int per, n;
      if (scanf("%lld %d %d", &cap, &per, &n) != 3) return 1;
      printf("%d\n", kvq::batch_items(cap, per, n));
      continue;
    }
    int items, n;
    if (scanf("%d %d", &items, &n) != 2) return 1;
    std::vector<int> t(n);
    long long total = 0;
    for (int& x : t) { if (scanf("%d", &x) != 1) return 1; total += x; }
    printf("%d\n", kvq::batch_split(total, items, n, [&](int s) { int c = 0; for (int x : t) c += (x + s - 1) / s; return c; }));
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("batch_splits")
    (d / "p.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", CSRC, str(d / "p.cpp"), "-o", str(d / "p")], check=True)

    def run(lines):
        r = subprocess.run([str(d / "p")], input="\n".join(lines), capture_output=True, text=True, check=True)
        return [int(x) for x in r.stdout.split()]
    return run


def count(tiles, s):
    return sum(-(-t // s) for t in tiles)


def test_the_splits_fit_and_are_near_the_shortest(ask):
    rng = random.Random(0)
    cases, lines = [], []
    for _ in range(500):
        n = rng.randrange(2, 129)
        items = n + rng.randrange(1, 5 * n)
        tiles = [0 if rng.random() < 0.1 else int(2 ** rng.uniform(0, rng.choice([3, 8, 15]))) for _ in range(n)]
        if rng.random() < 0.2:
            tiles = [1 << 20] + [1] * (n - 1)
        cases.append((items, tiles))
        lines.append(f"s {items} {n} " + " ".join(map(str, tiles)))
    for (items, tiles), s in zip(cases, ask(lines)):
        assert s >= 1 and count(tiles, s) <= items
        least = next(x for x in range(max(1, -(-sum(tiles) // items)), s + 1) if count(tiles, x) <= items)
        # steps of 1 + s / 64 from below: past the least by less than one, or the
        # sure length after 32 of them
        sure = -(-sum(tiles) // (items - len(tiles)))
        assert s <= least + 1 + s // 64 or s <= sure


def test_known_lengths(ask):
    # 4 sequences of 10 tiles for 8 splits: 5 tiles each; nothing to read: 1; one of
    # 100 among empty ones for 10: 10; 3, 3, 3 for 4 splits: 3
    assert ask(["s 8 4 10 10 10 10", "s 8 4 0 0 0 0", "s 10 4 0 100 0 0", "s 4 3 3 3 3"]) == [5, 1, 10, 3]


def test_waves(ask):
    # 608 CTAs, 8 heads: 76 splits a wave.  16 sequences want 64: one wave; 32 want
    # 128: two; 100 want 400, more than 4 waves' 304, which still exceed 100; 128
    # sequences of 32 heads x 2 row tiles: 38 <= 128, the host's plan.  One sequence,
    # and more than 128: the host's plan.
    assert ask(["i 608 8 16", "i 608 8 32", "i 608 8 100", "i 608 64 128", "i 608 8 1", "i 608 8 129"]) == [76, 152, 304, 0, 0, 0]
