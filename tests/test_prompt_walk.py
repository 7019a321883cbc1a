"""The walk over the tiles of packed prompts (csrc/pa_prompt_walk.cuh), compiled for the host.

A CTA of the bf16 prompt kernels looks up one index after another in one walk, in
ascending order, whichever indices the other CTAs leave to it: together they must find every
tile of every prompt once, and nothing at the indices behind the last tile.
"""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("walk") / "walk.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", f"-I{CUDA}/include",
                    "-I" + os.path.join(ROOT, "paged_kv_cache_335_b200", "csrc"), "-I" + os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "prompt_walk_host.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


def _walk(host, cu, total, max_len, block, group, per, rev, index):
    cu = np.asarray(cu, dtype=np.int32)
    index = np.asarray(index, dtype=np.int32)
    out = np.full((len(index), 4), -9, dtype=np.int32)
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    rc = host.prompt_walk(p(cu), len(cu) - 1, total, max_len, block, group, per, int(rev), p(index), len(index), p(out))
    assert rc >= 0, "the lanes of a warp parted"
    return [tuple(x) for x in out.tolist()], bool(rc)


def _count(n, block, group, per):
    return (-(-n // block) * group + per - 1) // per


BATCHES = [
    [2048] * 64, [1024] * 64, [700] * 64, [64] * 40,
    [1] * 33 + [5000],                       # the long one in the second 32
    [5000] * 3 + [1] * 40 + [3000, 0, 129],
    [random.Random(7).randint(1, 3000) for _ in range(48)],
    [random.Random(8).choice([0, 1, 127, 128, 129, 900]) for _ in range(70)],
    [300, 77], [0] * 40, [],
]


@pytest.mark.parametrize("lens", BATCHES, ids=range(len(BATCHES)))
@pytest.mark.parametrize("block,group,per,rev", [(128, 1, 2, True), (128, 4, 2, True), (128, 5, 2, True),
                                                 (256, 1, 1, False), (64, 1, 1, True)])
def test_every_tile_is_found_once(host, lens, block, group, per, rev):
    cu = np.cumsum([0] + lens)
    counts = [_count(n, block, group, per) for n in lens]
    tiles = sum(counts)
    rng = random.Random(len(lens) * block + group)
    ctas = 11
    mine = [[] for _ in range(ctas)]         # whichever CTA asks next gets the next index
    for u in range(tiles + 40):
        mine[u if u < ctas else rng.randrange(ctas)].append(u)
    found = {}
    for index in mine:
        got, bad = _walk(host, cu, int(cu[-1]), max(lens + [0]), block, group, per, rev, index)
        assert not bad
        for u, t in zip(index, got):
            if u >= tiles:
                assert t[0] == -1
                continue
            s, start, n, tile = t
            assert 0 <= s < len(lens) and (start, n) == (cu[s], lens[s]) and 0 <= tile < counts[s], (u, t)
            assert (s, tile) not in found, f"indices {found[s, tile]} and {u} both give tile {tile} of prompt {s}"
            found[s, tile] = u
    assert len(found) == tiles


def test_an_index_alone_gives_what_the_walk_gives(host):
    lens = [900, 0, 130] * 23
    cu = np.cumsum([0] + lens)
    index = list(range(0, 400, 3))
    got, _ = _walk(host, cu, int(cu[-1]), 900, 128, 2, 2, True, index)
    for u, t in zip(index, got):
        assert _walk(host, cu, int(cu[-1]), 900, 128, 2, 2, True, [u])[0] == [t]
    back, _ = _walk(host, cu, int(cu[-1]), 900, 128, 2, 2, True, index[::-1])
    assert back[::-1] == got


def test_bad_prompts_have_no_tile(host):
    for cu, total, longest, good in (([-1, 200, 250, 310], 310, 310, {1: 50, 2: 60}),
                                     ([0, 200, 250, 311], 310, 310, {0: 200, 1: 50}),
                                     ([0, 200, 250, 310], 310, 100, {1: 50, 2: 60}),
                                     ([0, 1] + [1] * 38 + [311], 310, 310, {0: 1})):
        got, bad = _walk(host, cu, total, longest, 64, 1, 1, True, range(20))
        assert bad
        want = sorted((s, t) for s, n in good.items() for t in range(-(-n // 64)))
        assert sorted((t[0], t[3]) for t in got if t[0] >= 0) == want


@pytest.mark.parametrize("cu,good", [
    ([0, 300, 0, 300], {0}),                             # the third prompt holds the first one's rows
    ([0, 200, 190, 310], {0}),
    ([0, 100, 500, 90, 95, 120, 130], {0, 5}),           # 100..500 lies outside; 90..95 and 95..120 come too early
    ([0, 10] + [10] * 30 + [310, 0, 200, 200, 310], {0, 31}),   # across the 32
    ([200, 310, 0, 100], {0}),
])
def test_prompts_that_overlap_an_earlier_one_have_no_tile(host, cu, good):
    """The grids are sized for disjoint prompts: total tokens / tile + prompts."""
    for block in (64, 128):
        got, bad = _walk(host, cu, 310, 310, block, 1, 1, True, range(100))
        assert bad
        want = sorted((s, t) for s in good for t in range(-(-(cu[s + 1] - cu[s]) // block)))
        assert sorted((t[0], t[3]) for t in got if t[0] >= 0) == want
        assert len(want) <= 310 // block + len(cu) - 1
