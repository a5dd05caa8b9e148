"""Plans of the shared-prefix decode for batches that do not fill their tiles: the own
keys of the requests that there are, not of as many as a tile could hold."""
import math
import os
import shutil

import pytest

from split_kv_mla_gb300 import build as mla_build
from split_kv_mla_gb300 import mla


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(mla_build.LIB):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("library not built and nvcc not available")
        mla_build.build()
    return mla.load()


def requests_of(t, per, rows):
    return t * 64 // per, (min(t * 64 + 64, rows) - 1) // per


@pytest.mark.parametrize("batch", [1, 2, 3, 5, 8, 31, 64, 100])
@pytest.mark.parametrize("per", [1, 3, 8, 16, 24, 40, 64, 96, 128])
@pytest.mark.parametrize("prefix,own", [(1, 1), (300, 20), (300, 129), (1000, 1000), (16384, 4000),
                                        (8192, 8192), (200, 0)])
def test_no_more_parts_than_blocks(batch, per, prefix, own):
    p = mla.mla_prefix_decode_plan(batch, 1, per, prefix, batch * own, 152)
    rows, shared, mine = batch * per, -(-prefix // 128), -(-own // 128) * p.joined
    blocks = []
    for t in range(p.tiles):
        b0, b1 = requests_of(t, per, rows)
        blocks.append(shared + (b1 - b0 + 1) * mine)
    if p.splits:
        assert p.splits <= max(blocks)
    else:
        assert p.ctas <= sum(blocks)


@pytest.mark.parametrize("seed", range(20))
def test_pairs_of_tiles_and_requests(seed):
    # the closed form that the plan uses: the tiles' and the requests' borders cut the rows
    # into tiles + batch - 1 pieces, less the borders that they share
    import random
    rng = random.Random(seed)
    per, batch = rng.randrange(1, 300), rng.randrange(1, 200)
    rows = batch * per
    tiles = -(-rows // 64)
    pairs = 0
    for t in range(tiles):
        b0, b1 = requests_of(t, per, rows)
        pairs += b1 - b0 + 1
    assert pairs == tiles + batch - 1 - (rows - 1) // math.lcm(per, 64)


@pytest.mark.parametrize("batch,heads,prefix,own", [
    # measured, tiles' own blocks (the choice) against a launch of their own: 21.8 against
    # 35.7 us, 21.8 / 34.8, 24.6 / 34.4, 24.7 / 36.5, 17.6 / 28.5
    (1, 1, 16384, 4000), (1, 8, 8192, 8192), (2, 1, 8192, 8192), (2, 8, 16384, 4000),
    (1, 1, 1000, 1000)])
def test_few_requests_with_long_own_keys_join(batch, heads, prefix, own):
    assert mla.mla_prefix_decode_plan(batch, 1, heads, prefix, batch * own, 152).joined == 1


def test_a_merge_of_few_partials():
    # 64 parts of two blocks 21.7 us, 128 of one 24.6: few rows' merges take 80 at a time
    p = mla.mla_prefix_decode_plan(1, 1, 16, 8192, 8192, 152)
    assert (p.joined, p.ctas, p.splits) == (1, 64, 64)
