"""CPU checks of which kernels the sizes in the GPU tests of mxq_linear_ce_* take: each kernel is run by some
test, so that a rule that moves cannot leave one without, and the sizes that are listed for a kernel take it."""
import pytest

import ce_kernels
import test_gpu_linear_ce as bounded
import test_gpu_linear_ce_exact as exact
import test_gpu_linear_ce_plans as plans
import test_gpu_linear_ce_rounding as rounding
import test_gpu_linear_ce_tiles as tiles


def every():
    return {(name, tile, cut) for name, of in ce_kernels.OF.items() for tile in of
            for cut in ((False, True) if name != "dw" else (False,))}


def taken(shapes, piece=ce_kernels.SHIPPED):
    return {(name, *ce_kernels.kernels(*s, piece)[name]) for s in shapes for name in ce_kernels.OF}


def test_every_kernel_is_tested():
    # against the formulas with bounds, and on sums that are exact in any order
    assert taken(bounded.SHAPES + tiles.SHAPES + [(2600, 544, 4160)]) == every()
    assert taken(exact.SHAPES + tiles.SHAPES + list(plans.LARGE)) == every()


def test_every_tile_of_dw_keeps_targets():
    assert {k for k in taken(rounding.SHAPES) if k[0] == "dw"} == {k for k in every() if k[0] == "dw"}


@pytest.mark.parametrize("shape,want,piece", [(s, w, ce_kernels.SHIPPED) for s, w in plans.LARGE.items()] +
                         [(s, w, ce_kernels.LOOP) for s, w in plans.PIECES.items()], ids=str)
def test_listed_for(shape, want, piece):
    got = ce_kernels.kernels(*shape, piece)
    assert {k: got[k] for k in want} == want


def test_what_the_library_takes_for_large_steps():
    got = ce_kernels.kernels(8192, 4096, 128256)
    assert got["pieces"] == 8 and got["slabs"] == 1
    # the kernels that this takes over several pieces are those that the sizes above run over several pieces
    seen = taken([s for s, w in plans.LARGE.items() if w.get("pieces", 1) > 1])
    for name in ("dz", "dx", "dw"):
        assert (name, *got[name]) in seen
