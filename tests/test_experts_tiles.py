"""Which tile the expert stage's products run on, without a GPU: the rule against the kernels that are built."""
import os
import re

import pytest

import combine_moe_get_amd as mg
from tests import _isa, _tiles

PRODUCTS = [(mg.EXPERTS_FORWARD, t, a) for t in (mg.ROWS_BF16, mg.ROWS_INT8, mg.ROWS_MXFP4)
            for a in (mg.ACT_NONE, mg.ACT_SWIGLU)]
PRODUCTS += [(op, mg.ROWS_BF16, mg.ACT_NONE) for op in (mg.EXPERTS_DGRAD, mg.EXPERTS_WGRAD)]


def _selected():
    """{(row type, product, gate, tile, whole words of scales)} over a grid of sizes."""
    found = set()
    for rows in (1, 8, 100, 400, 1000, 2000, 4000, 8000, 16000, 32768, 200000):
        for E in (1, 2, 4, 8, 16, 32, 64, 256):
            for k in (32, 416, 1024, 2048, 4096, 7168):
                for n in (48, 512, 1024, 2048, 4096, 8192):
                    s = mg.make_experts_shape(rows, E, k, n)
                    for op, ty, act in PRODUCTS:
                        wide = ty != mg.ROWS_MXFP4 or k % 128 == 0
                        found.add((ty, op, act, mg.experts_tile(s, op, ty, act), wide))
    return found


@pytest.mark.skipif(not os.path.exists(_isa.OBJDUMP) or not os.path.exists(mg.LIB_PATH),
                    reason="needs llvm-objdump and the built library")
def test_every_kernel_that_is_built_is_selected_by_some_size():
    built = set()
    for name in _isa.kernels():
        m = re.search(r"experts_kernel<(\d), (\d), (true|false), (true|false), (\d+), (\d+), \d, \d, (\d), \w+, (true|false)>",
                      name)
        if m:
            ty, op, gate, _, bm, bn, stages, wide = m.groups()
            built.add((int(ty), int(op), int(gate == "true"), (int(bm), int(bn), int(stages)), wide == "true"))
    assert built == _selected()


def test_tile_refuses():
    s = mg.make_experts_shape(64, 8, 64, 24)
    for op, ty, act in PRODUCTS:
        assert mg.experts_tile(s, op, ty, act)[0] in (16, 64)
    for bad in ((3, 0, 0), (-1, 0, 0), (0, 3, 0), (0, 0, 2), (mg.EXPERTS_DGRAD, 1, 0), (mg.EXPERTS_WGRAD, 0, 1)):
        with pytest.raises(mg.MoeGetError):
            mg.experts_tile(s, *bad)
    with pytest.raises(mg.MoeGetError):
        mg.experts_tile(mg.make_experts_shape(64, 8, 72, 24), 0, mg.ROWS_INT8)


@pytest.mark.parametrize("case", _tiles.CASES, ids=_tiles.name)
def test_sizes_that_are_run_for_a_tile_select_it(case):
    op, ty, act, tile, E, mean, k, n = case
    assert mg.experts_tile(_tiles.rows_of(E, mean).shape(k, n), op, ty, act) == tile


def test_every_tile_has_sizes_that_are_run():
    run = {(ty, op, act, tile, ty != mg.ROWS_MXFP4 or k % 128 == 0) for op, ty, act, tile, _, _, k, _ in _tiles.CASES}
    assert run == _selected()
