"""How the attention of chunks shares segments out among its blocks (csrc/chunk_plan.h), without a GPU: the header is compiled
with g++ through tests/chunk_plan_driver.cpp, and its choice compared with the tiles that the busiest block gets either way."""
import os
import shutil
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "speculative_decoding_token_temp_gb300", "csrc")
BLOCKS, SEG, JOIN = 152, 4, 9  # blocks of a GB300's wave, tiles that a segment's ends and the joining count for


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path_factory.mktemp("chunk") / "driver")
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "chunk_plan_driver.cpp"), "-o", exe], check=True, capture_output=True)

    def query(lines):
        out = subprocess.run([exe], input="\n".join(" ".join(str(int(x)) for x in q) for q in lines) + "\n", capture_output=True, text=True, check=True)
        return [bool(int(x)) for x in out.stdout.split()]
    return query


def both(tiles, heads):
    """(tiles of the busiest block when segments stay whole, when the line is cut; the query) of row blocks of these lengths."""
    each = np.sort(np.repeat(np.asarray(tiles), heads))[::-1] + SEG
    dealt = np.zeros(-(-len(each) // BLOCKS) * BLOCKS, dtype=np.int64)
    dealt[:len(each)] = each
    dealt = dealt.reshape(-1, BLOCKS)
    dealt[1::2] = dealt[1::2, ::-1].copy()
    whole, line = int(dealt.sum(0).max()), int(each.sum())
    busiest = whole if len(each) <= 64 * BLOCKS else 0
    return whole, line // BLOCKS + SEG + JOIN, (len(each), BLOCKS, busiest, int(max(tiles)), line, SEG)


def test_one_long_segment_among_many_short_ones_is_cut(choose):
    """About 1250 sequences of one token behind a few, one behind a million, at 8 kv heads: more than 64 segments a block."""
    whole, cut, query = both([1] * 1250 + [7813], 8)
    assert query[0] > 64 * BLOCKS and whole > 8 * cut
    assert choose([query]) == [False]


def test_many_short_segments_stay_whole(choose):
    queries = [both([1] * 1300, 8)[2], both([3] * 40000, 1)[2], both(list(range(1, 64)) * 40, 8)[2]]
    assert all(q[0] > 64 * BLOCKS for q in queries)
    assert choose(queries) == [True] * 3


def test_the_choice_is_never_much_worse_than_the_other(choose):
    """Past what is added up, whole segments leave the busiest block at most the longest one, an eighth of its share, more."""
    rng = np.random.default_rng(5)
    cases = []
    for _ in range(400):
        heads = int(rng.choice([1, 2, 4, 8]))
        n = int(64 * BLOCKS // heads * rng.choice([0.02, 0.2, 0.9, 1.1, 2.0])) + 1
        tiles = np.maximum(1, rng.choice([1, 2, 5, 20, 100]) * np.exp(rng.normal(0, rng.choice([0.1, 0.5, 1, 2]), n)))
        tiles[:int(rng.choice([1, 3, 20, 100]))] *= rng.choice([1, 3, 10, 100, 1000])
        cases.append(both(np.minimum(tiles, 8192).astype(int), heads))
    for (whole, cut, query), is_whole in zip(cases, choose([q for _, _, q in cases])):
        assert (whole if is_whole else cut) <= 1.125 * min(whole, cut), query
