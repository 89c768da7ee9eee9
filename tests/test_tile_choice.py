"""The estimate by which the tiled products choose their tile size (host only)."""
import os
import random
import re
import shutil

import pytest

import tile_choice


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not installed")
    return tile_choice.Tiles(tmp_path_factory.mktemp("tiles"))


def draw(rng):
    log = lambda lo, hi: int(lo * (hi / lo) ** rng.random())  # noqa: E731
    return log(1, 60000), 64 * log(1, 130), 32 * log(1, 260)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_tile_size_is_chosen(tiles, dtype):
    """No size that is compiled for a launch is one that no call of it takes."""
    rng = random.Random(7)
    asked = [tile_choice.launches(dtype, *draw(rng)) for _ in range(10000)]
    for launch in asked[0]:
        assert set(tiles.ask([q[launch] for q in asked])) == set(tiles.sizes(dtype)), launch


def test_tiles_are_the_kernels(tiles):
    """The sizes of the cost tables, in order, are those of the kernels' configurations."""
    src = open(os.path.join(tile_choice.CSRC, "tile_gemm.h")).read()
    for dtype, c in (("bf16", "uint16_t"), ("f32", "float")):
        found = re.findall(r"struct TileCfg<%s, (\d), TA, TB> \{ typedef Cfg<%s, (\d+), (\d+)," % (c, c), src)
        assert [int(i) for i, _, _ in found] == list(range(len(found)))
        assert [(int(m), int(n)) for _, m, n in found] == tiles.sizes(dtype)
