"""The index arithmetic of the append to an 8-bit cache (csrc/append8_places.h), compiled for the host: which page of
which sequence each unit of the kernel belongs to, for offsets as they should be and for offsets that decrease."""
import ctypes
import os
import random
import subprocess

import pytest

from tests.conftest import ROOT

SOURCE = """
#include "append8_places.h"
extern "C" void unit(uint32_t place, int B, int T, int page, const int* cu, const int* lens, int* out) {
  const int b = fa::search_places(B, [&](int lo, int step, int end) {
    int n = 0;  // as the lanes of a warp count
    for (int lane = 0; lane < 32; ++lane) {
      const int i = lo + (lane + 1) * step - 1;
      n += i < end && fa::first_place(cu[i], page, i) <= place;
    }
    return n;
  });
  out[0] = b;
  if (b < 0 || b >= B) return;
  const fa::Piece x = fa::piece_of(place, b, cu[b], cu[b + 1], lens[b], T, page);
  out[1] = x.at, out[2] = x.s0, out[3] = x.s1, out[4] = x.alive, out[5] = x.early;
}
"""


@pytest.fixture(scope="module")
def units(tmp_path_factory):
    d = tmp_path_factory.mktemp("places")
    src, lib = d / "places.cpp", d / "places.so"
    src.write_text(SOURCE)
    csrc = os.path.join(ROOT, "exact_attention_forward_02_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", csrc, str(src), "-o", str(lib)],
                   check=True)
    f = ctypes.CDLL(str(lib)).unit
    f.argtypes = [ctypes.c_uint32] + [ctypes.c_int] * 3 + [ctypes.POINTER(ctypes.c_int)] * 3

    def all_units(cu, lens, T, page):
        """(b, at, s0, s1, alive, early) of every place that the launch has."""
        B = len(lens)
        c, n, out = (ctypes.c_int * (B + 1))(*cu), (ctypes.c_int * B)(*lens), (ctypes.c_int * 6)()
        got = []
        for place in range(T // page + 2 * B):
            out[:] = [0] * 6
            f(place, B, T, page, c, n, out)
            got.append(tuple(out))
        return got
    return all_units


def pages_of(cu, lens, T, page, b):
    """{page of sequence b: slots that get new tokens}, from the definition, and whether tokens lie before position 0."""
    n = cu[b + 1] - cu[b]
    if cu[b] < 0 or n <= 0 or cu[b + 1] > T:
        return {}, False
    want = {}
    for pos in range(max(lens[b] - n, 0), max(lens[b], 0)):
        want.setdefault(pos // page, []).append(pos % page)
    return {at: (s[0], s[-1] + 1) for at, s in want.items()}, lens[b] < n


def check(got, cu, lens, T, page, complete):
    """Every unit that works is one of its sequence's own pages, none stands twice; `complete`: none is missing."""
    seen = {}
    for b, at, s0, s1, alive, _ in got:
        assert -1 <= b < len(lens)
        if not alive:
            continue
        assert at >= 0 and (b, at) not in seen
        assert pages_of(cu, lens, T, page, b)[0][at] == (s0, s1)
        seen[b, at] = 1
    if complete:
        for b in range(len(lens)):
            want, early = pages_of(cu, lens, T, page, b)
            assert all((b, at) in seen for at in want)
            assert sum(x[5] for x in got if x[0] == b) == early


def test_decreasing_offsets_never_ask_for_an_entry_before_the_table(units):
    """Offsets [0, 900, 1000, 0, 10] of 1000 rows, pages of 16: the search for places 6 to 57 ends at sequence 1, whose
    own rows are in order but whose first place is 58."""
    cu, lens, T, page = [0, 900, 1000, 0, 10], [900, 100, 0, 10], 1000, 16
    got = units(cu, lens, T, page)
    assert any(b == 1 and place < 58 for place, (b, *_) in enumerate(got))
    check(got, cu, lens, T, page, False)


@pytest.mark.parametrize("page", [8, 16, 384])
def test_offsets_in_any_order(units, page):
    rng = random.Random(page)
    for _ in range(300):
        T, B = rng.randint(1, 3000), rng.choice([1, 2, 5, 31, 33, 70])
        cu = [rng.randint(-20, T + 20) for _ in range(B + 1)]
        if rng.random() < 0.5:
            cu = sorted(cu)
            cu[rng.randrange(B + 1)] = rng.randint(0, T)
        lens = [rng.choice([0, -5, rng.randint(0, 4000), 1 << 30]) for _ in range(B)]
        got = units(cu, [min(n, 5000) for n in lens], T, page)
        check(got, cu, [min(n, 5000) for n in lens], T, page, False)


@pytest.mark.parametrize("page", [8, 16, 64, 128, 384])
def test_every_page_has_its_unit(units, page):
    rng = random.Random(page)
    for _ in range(150):
        B = rng.choice([1, 2, 5, 32, 33, 64])
        new = [rng.choice([0, 1, 1, 3, rng.randint(0, 3 * page)]) for _ in range(B)]
        cu = [rng.randint(0, 40)]
        for n in new:
            cu.append(cu[-1] + n)
        lens = [max(0, n + rng.randint(-3 if rng.random() < 0.1 else 0, 2 * page)) for n in new]
        T = cu[-1] + rng.randint(0, 30)
        check(units(cu, lens, T, page), cu, lens, T, page, True)


def test_lengths_near_the_end_of_32_bits(units):
    top = 0x7fffffff
    for lens in ([top], [-top - 1], [1 << 30]):
        for b, at, s0, s1, alive, early in units([0, 20], lens, 20, 8):
            assert early in (0, 1)
            if alive:
                assert 0 <= at * 8 + s0 < at * 8 + s1 <= lens[0] and lens[0] - 20 <= at * 8 + s0
