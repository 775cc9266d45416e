"""CPU checks of the note that a CTA of the attention leaves for the join:
every note of a call is followed, and none whose numbers would lead outside
the call's tensors or the join's tables; and of a part's weight there.  The
checks are compiled from the kernel's own header."""
import ctypes
import math
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "tree_verified_speculative_gb300", "csrc")
SRC = """
#include "join_note.h"
extern "C" int usable(const int *n, int cta, int n_cta, int n_req, int Hk, int n_pair, int N) {
  mfd::Cut c;
  c.has[0] = n[0]; c.has[1] = n[1]; c.reach = n[2]; c.q = n[3]; c.h = n[4]; c.pair = n[5]; c.nn = n[6];
  return mfd::cut_usable(c, cta, n_cta, n_req, Hk, n_pair, N);
}
extern "C" float weight(int slot, float w, float inv) { return mfd::join_weight(slot, w, inv); }
extern "C" float tiny_weight() { return mfd::TINY_WEIGHT; }
extern "C" int note_bytes() { return (int)sizeof(mfd::Cut); }
extern "C" int empty() { const mfd::Cut c{}; return c.has[0] | c.has[1] | c.reach | c.q | c.h | c.pair | c.nn; }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("note")
    src, out = str(d / "note.cpp"), str(d / "note.so")
    with open(src, "w") as f:
        f.write(SRC)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, src, "-o", out], check=True)
    so = ctypes.CDLL(out)
    so.weight.argtypes, so.weight.restype = [ctypes.c_int, ctypes.c_float, ctypes.c_float], ctypes.c_float
    so.tiny_weight.restype = ctypes.c_float
    return so


def usable(lib, note, *call):
    return bool(lib.usable((ctypes.c_int * 7)(*note), *call))


def test_an_empty_note_is_not_followed(lib):
    assert lib.note_bytes() == 28 and lib.empty() == 0
    assert not usable(lib, [0] * 7, 0, 152, 4, 8, 3, 129)


def test_notes_of_random_lines_are_followed(lib):
    """A line of items cut by borders: the CTA that holds an item's first tiles
    notes it, with the CTAs up to the one with the item's last place."""
    rng = random.Random(1)
    n = 152
    for _ in range(50):
        R, Hk, pairs, N = rng.randint(1, 9), rng.randint(1, 8), rng.randint(1, 5), rng.randint(1, 300)
        items = [(q, h, i, rng.randint(6, 400)) for q in range(R) for h in range(Hk) for i in range(pairs)]
        total = sum(x[3] for x in items)
        x = 0
        for q, h, i, cost in items:
            first, last = ((x + 1) * n - 1) // total, ((x + cost) * n - 1) // total
            if first != last:
                assert usable(lib, [0, 1, last - first + 1, q, h, i, rng.randint(1, N)], first, n, R, Hk, pairs, N)
            x += cost


def test_stale_scratch_is_not_followed(lib):
    """Whatever the scratch holds, a note that is followed stays inside."""
    rng = random.Random(2)
    edge = [-2 ** 31, -1, 0, 1, 2, 7, 8, 151, 152, 153, 0x5A5A5A5A, 2 ** 31 - 1, -0x5A5A5A5B]
    followed = 0
    for _ in range(200000):
        n_cta, R, Hk, pairs, N = rng.choice([1, 8, 152]), rng.randint(1, 9), rng.randint(1, 8), rng.randint(1, 5), rng.randint(1, 9)
        cta = rng.randrange(n_cta)
        note = [rng.choice(edge) for _ in range(7)]
        if usable(lib, note, cta, n_cta, R, Hk, pairs, N):
            followed += 1
            _, _, reach, q, h, pair, nn = note
            assert 1 <= reach and cta + reach <= n_cta  # entries of the join's tables, and notes read
            assert 0 <= q < R and 0 <= h < Hk and 0 <= pair < pairs and 1 <= nn <= N  # rows of the output
    assert followed > 0
    good = [0, 1, 3, 1, 1, 1, 5]
    assert usable(lib, good, 10, 152, 2, 2, 2, 5)
    for at, bad in ((2, 143), (2, 0), (2, -1), (3, 2), (3, -1), (4, 2), (4, -1), (5, 2), (5, -1), (6, 6), (6, 0), (6, -1)):
        assert not usable(lib, good[:at] + [bad] + good[at + 1:], 10, 152, 2, 2, 2, 5), (at, bad)


def test_an_absent_part_has_no_weight(lib):
    """Whatever a row's sum is, a part that is not there (slot -1) has weight
    zero and is not read; a part that is there keeps a NaN."""
    inf, nan = float("inf"), float("nan")
    for w in (0.0, 1.0, nan, inf, lib.tiny_weight()):
        for inv in (0.0, 0.5, nan, inf, -inf):
            assert lib.weight(-1, w, inv) == 0.0, (w, inv)
    assert lib.weight(0, 0.5, 0.5) == 0.25 and lib.weight(7, 1.0, 0.0) == 0.0
    assert math.isnan(lib.weight(3, 0.0, nan)) and math.isnan(lib.weight(3, nan, 1.0)) and math.isnan(lib.weight(3, 1.0, nan))
    tiny = lib.tiny_weight()
    assert tiny < 0 and lib.weight(3, tiny, 0.5) == tiny
