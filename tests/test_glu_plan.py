"""How a gated feed-forward call is cut, as the calls themselves decide it (CPU)."""
import pytest

import attention_qkv_gemm_gb300 as pkg
from attention_qkv_gemm_gb300 import build as libbuild
from tests.glu_forms import WANTED, reached


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return pkg.load()


# CTAs, pairs and clusters of 2, 4 and 8 that a GPU of 152 SMs may run at once: a cluster stays within
# a processing cluster, whose SMs need not be a multiple of it
@pytest.mark.parametrize("units", [(152, 76, 76, 38, 18), (152, 74, 74, 36, 16), (148, 72, 72, 36, 17)])
def test_the_tests_sizes_reach_every_form_in_every_mode(units):
    assert reached(units) == WANTED


@pytest.mark.parametrize("units", [(152, 76, 76, 38, 18), (152, 76, 0, 0, 0), (1, 1, 0, 0, 0)])
def test_every_size_is_cut_within_the_kernels_limits(units):
    """Tiles of 16 to 128 output columns of each product (32 to 256 of one), pairs' in steps of 16 (32),
    every column covered, no more clusters than tiles at once."""
    import random
    rng = random.Random(0)
    for _ in range(3000):
        kind = rng.choice([pkg.TFL_BF16, pkg.TFL_E4M3])
        step = 16 if kind == pkg.TFL_E4M3 else 8
        d, f = (step * rng.randint(1, 4 ** rng.randint(1, 6)) for _ in range(2))
        tokens, part = rng.randint(1, 4 ** rng.randint(1, 8)), 0 if kind == pkg.TFL_E4M3 else rng.randint(0, 3)
        form, bno, tiles, at_once = pkg.tfl_selftest_glu_plan(d, f, kind, part, tokens, units)
        if form == pkg.TFL_GLU_FORM_FEW:
            assert part == 0 and tokens <= 16
            continue
        two = part < 2
        rows, cols = (f, d) if part == 3 else (tokens, d if part == 2 else f)
        pairs = form >= pkg.TFL_GLU_FORM_PAIR
        columns = 2 * bno if two else bno
        assert 32 <= columns <= 256 and columns % (32 if pairs else 16) == 0
        assert (form == pkg.TFL_GLU_FORM_WIDE) == (pairs and columns == 256)
        height = 256 if pairs else 128
        assert tiles == -(-rows // height) * -(-cols // bno) * (2 if part == 3 else 1)
        assert 1 <= at_once and (form != pkg.TFL_GLU_FORM_SHARED or tiles <= at_once)
        assert not pairs or rows > 128


@pytest.mark.parametrize("args", [(0, 64, 2, 0, 1), (64, 0, 2, 0, 1), (64, 64, 0, 0, 1), (64, 64, 2, 4, 1), (64, 64, 2, -1, 1),
                                  (64, 64, 3, 1, 1), (64, 64, 2, 0, 0), (64, 64, 2, 0, 1 << 31), ((1 << 24) + 8, 64, 2, 0, 1),
                                  (64, (1 << 24) + 8, 2, 0, 1)])
def test_refusals(args):
    with pytest.raises(pkg.TflError) as e:
        pkg.tfl_selftest_glu_plan(*args, (152, 76, 76, 38, 18))
    assert e.value.code == pkg.TFL_ERR_INVALID_ARG and str(e.value)
