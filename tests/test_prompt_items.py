"""The search of an item among ragged sequences, without a GPU: the kernel's own code, its warp's lanes
played by a loop."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Reads B, T, max_len, Hkv, per, n, the B + 1 starts, n item numbers; writes an item a line.
MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "prompt_items.h"

struct Lanes {
  const kvq::PromptSeqs& s;
  unsigned longer(int b0, int than) const {
    unsigned m = 0;
    bool wrong = false;
    for (int i = 0; i < 32; ++i)
      if (kvq::prompt_length(s, b0 + i, &wrong) > than) m |= 1u << i;
    return m;
  }
  int nth(unsigned m, int r) const {
    if (r < 0) std::abort();
    for (int i = 0; i < 32; ++i)
      if ((m >> i & 1u) && r-- == 0) return i;
    return -1;
  }
};

int main() {
  int B, max_len, Hkv, per, n;
  long long T;
  if (std::scanf("%d %lld %d %d %d %d", &B, &T, &max_len, &Hkv, &per, &n) != 6) return 1;
  int* start = new int[B + 1];                 // by itself, for the address checks
  for (int b = 0; b <= B; ++b) if (std::scanf("%d", start + b) != 1) return 1;
  const kvq::PromptSeqs s = {start, T, B, max_len, Hkv, per};
  const Lanes lanes = {s};
  int longest = 0, wrongs = 0;
  for (int b = 0; b < B; ++b) {
    bool wrong = false;
    const int len = kvq::prompt_length(s, b, &wrong);
    longest = len > longest ? len : longest;
    wrongs += wrong;
  }
  kvq::PromptSearch<Lanes> search(s, lanes, longest);
  std::printf("%d\n", wrongs);
  for (int i = 0; i < n; ++i) {
    long long w;
    if (std::scanf("%lld", &w) != 1) return 1;
    const kvq::PromptItem it = search.find(w);
    std::printf("%d %d %d %d\n", it.t0, it.p0, it.end, it.g);
  }
  delete[] start;
}
"""


@pytest.fixture(scope="module")
def find(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("wants g++")
    d = tmp_path_factory.mktemp("items")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-I" + os.path.join(ROOT, "int4_quantized_paged_gb300", "csrc"), str(d / "main.cpp"), "-o",
                    str(d / "find")], check=True)

    def run(starts, T, max_len, Hkv, per, order):
        text = " ".join(map(str, [len(starts) - 1, T, max_len, Hkv, per, len(order), *starts, *order]))
        r = subprocess.run([str(d / "find")], input=text, capture_output=True, text=True, timeout=60,
                           env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
        assert r.returncode == 0, r.stderr[-2000:]
        lines = r.stdout.splitlines()
        return int(lines[0]), [tuple(map(int, x.split())) for x in lines[1:]]
    return run


def _lengths(starts, T, max_len):
    """Tokens of each sequence that are computed, and how many sequences that leaves tokens out of."""
    lens, wrong = [], 0
    for s, e in zip(starts, starts[1:]):
        bad = s < 0 or e < s or e > T
        lens.append(0 if bad else min(e - s, max_len))
        wrong += bad or e - s > max_len
    return lens, wrong


def _items(starts, T, max_len, Hkv, per):
    lens, wrong = _lengths(starts, T, max_len)
    items = []
    for q in reversed(range(-(-max(lens, default=0) // per))):
        for s, n in zip(starts, lens):
            if n > q * per:
                items += [(s, q * per, min(n, (q + 1) * per), g) for g in range(Hkv)]
    return wrong, items


CASES = [
    # starts, T, max_len, Hkv, per
    ([0, 1], 1, 1, 1, 256),
    ([0, 0, 0], 5, 10, 2, 64),
    ([3, 203, 204, 268, 268, 333, 462, 479, 607, 607, 940], 1090, 333, 4, 64),
    ([0, 16384], 16384, 16384, 8, 64),
    ([0, 300, 320], 320, 130, 2, 32),                        # past the caller's bound
    ([-5, 95, 150], 150, 150, 2, 32),
    ([0, 200, 150], 150, 150, 2, 32),
    ([0, 100, 2 ** 31 - 1], 150, 150, 2, 32),
    ([0, 100, -2 ** 31], 150, 150, 2, 32),
    ([2 ** 31 - 1, -2 ** 31, 7], 150, 150, 2, 32),
    ([0, 140, 10, 150], 150, 150, 1, 32),                    # two sequences over the same tokens
]


def _ragged(seed):
    r = random.Random(seed)
    starts = [r.randint(0, 9)]
    for _ in range(r.choice([1, 31, 32, 33, 64, 70, 200])):
        starts.append(starts[-1] + r.choice([0, 1, r.randint(0, 40), r.randint(0, 900)]))
    return starts, starts[-1] + r.randint(0, 3), r.choice([900, 500]), r.choice([1, 2, 8]), r.choice([16, 64, 256])


@pytest.mark.parametrize("order", ["up", "down", "any", "two"])
@pytest.mark.parametrize("case", [pytest.param(c, id=f"case{i}") for i, c in enumerate(CASES)] +
                         [pytest.param(_ragged(s), id=f"ragged{s}") for s in range(12)])
def test_items_are_found_in_every_order(find, case, order):
    """Nothing says in which order the launches of a grid are cancelled."""
    wrong, want = _items(*case)
    n = len(want) + 3                                        # and none behind the last
    ws = list(range(n))
    if order == "down":
        ws.reverse()
    elif order == "any":
        random.Random(n).shuffle(ws)
        ws += ws[:5]
    elif order == "two":                                     # behind the last and back
        ws = [w for i in range(n) for w in (n + i, i)]
    got_wrong, got = find(*case, ws)
    assert got_wrong == wrong
    for w, it in zip(ws, got):
        assert (it == want[w]) if w < len(want) else (it[1] < 0), w
