"""How the key side of the local attention backward divides its work (csrc/rglru_shares.h, compiled here for the
host, no GPU): every part that is summed has been written, whatever the lengths are."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gated_linear_recurrence_conv1d_amd", "csrc")
SOURCE = """
#include "rglru_shares.h"
using namespace rglru::attn;
extern "C" {
int row_blocks_(int K0, int len, int window, int sinks) { return row_blocks(K0, len, window, sinks); }
int share_count_(long long items, int groups) { return share_count(items, groups); }
long long share_lo_(long long items, int n, int w) { return share_lo(items, n, w); }
int share_of_(long long items, int n, long long i) { return share_of(items, n, i); }
int own_() { return kOwn; }
int blk_() { return kBlk; }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("shares")
    (d / "shares.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-I" + CSRC, "-o",
                    str(d / "shares.so"), str(d / "shares.cpp")], check=True)
    lib = ctypes.CDLL(str(d / "shares.so"))
    ll = ctypes.c_longlong
    lib.share_count_.argtypes = [ll, ctypes.c_int]
    lib.share_lo_.argtypes, lib.share_lo_.restype = [ll, ctypes.c_int, ctypes.c_int], ll
    lib.share_of_.argtypes = [ll, ctypes.c_int, ll]
    return lib


def entries(lib, T, group, Hkv, W, S, lens):
    """Items of each (key/value head, sequence, key block)."""
    return [lib.row_blocks_(K0, n, W, S) * group for n in lens for K0 in range(0, T, lib.own_())] * Hkv


def unwritten(lib, items, n):
    """Parts that the sum reads and no workgroup writes, when n workgroups take part: workgroup w walks its share
    block by block and writes a part of each block that it has not whole, as first (its block's first item is
    among them) or not; the sum reads, of a block that several have, the first's part and the others'."""
    total = sum(items)
    first = [0]
    for m in items:
        first.append(first[-1] + m)
    written, whole = set(), set()
    for w in range(n):
        pos, hi = lib.share_lo_(total, n, w), lib.share_lo_(total, n, w + 1)
        while pos < hi:
            e = max(i for i in range(len(items)) if first[i] <= pos and items[i])
            i0 = pos - first[e]
            i1 = min(items[e], i0 + hi - pos)
            if i1 - i0 == items[e]:
                whole.add(e)
            else:
                written.add((w, e, i0 == 0))
            pos += i1 - i0
        assert len([x for x in written if x[0] == w]) <= 2  # the workspace has two places for each
        assert len([x for x in written if x[0] == w and x[2]]) <= 1
    missing = 0
    for e, m in enumerate(items):
        if not m:
            continue
        a, b = lib.share_of_(total, n, first[e]), lib.share_of_(total, n, first[e + 1] - 1)
        assert 0 <= a <= b < n
        assert (a == b) == (e in whole)
        if a != b:
            missing += sum((w, e, w == a) not in written for w in range(a, b + 1))
    return missing


SHORT = [  # T, group, Hkv, window, sinks, lens
    (2048, 1, 1, 1024, 0, [100]),
    (2048, 10, 1, 1024, 0, [100]),
    (2048, 10, 1, 1024, 4, [300]),
    (2048, 10, 1, 1024, 0, [64] * 4),
    (512, 4, 1, 256, 0, [512] + [20] * 7),
    (2048, 1, 3, 64, 0, [0, 1, 0]),
]


@pytest.mark.parametrize("T,group,Hkv,W,S,lens", SHORT)
def test_short_lengths(lib, T, group, Hkv, W, S, lens):
    items = entries(lib, T, group, Hkv, W, S, lens)
    assert unwritten(lib, items, lib.share_count_(sum(items), 256)) == 0
    # with the launch's number instead, whatever the items are, parts would be missing
    if sum(items) > 3:
        assert unwritten(lib, items, 256) > 0


def test_any_lengths(lib):
    rng = random.Random(7)
    for _ in range(300):
        T, B = rng.choice([1, 31, 128, 129, 500, 2048]), rng.randint(1, 5)
        lens = [rng.choice([0, 1, rng.randint(0, T), min(T, 40), T]) for _ in range(B)]
        items = entries(lib, T, rng.choice([1, 2, 5]), rng.choice([1, 2]), rng.choice([1, 7, 128, 1024, T]),
                        rng.choice([0, 1, 70, T]), lens)
        if sum(items):
            n = lib.share_count_(sum(items), rng.choice([1, 3, 64, 255, 256]))
            assert unwritten(lib, items, n) == 0
            assert all(lib.share_lo_(sum(items), n, w) < lib.share_lo_(sum(items), n, w + 1) for w in range(n))


def test_row_blocks(lib):
    """Against the definition: 32-row blocks with a row that sees one of the 128 keys."""
    own, blk = lib.own_(), lib.blk_()
    rng = random.Random(3)
    for _ in range(200):
        n, W, S = rng.randint(0, 700), rng.choice([1, 2, 33, 300, (1 << 31) - 1]), rng.choice([0, 1, 128, 200, 700])
        K0 = own * rng.randint(0, 5)
        sees = {t // blk for t in range(K0, n) for u in (K0, min(K0 + own - 1, n - 1, t))
                if u <= t and (u > t - W or u < S)}
        assert lib.row_blocks_(K0, n, W, S) == len(sees), (K0, n, W, S)
