"""Which kernel a call of the layer norm takes, as the calls themselves decide it (CPU)."""
import random

import pytest

import attention_qkv_gemm_gb300 as pkg
from attention_qkv_gemm_gb300 import build as libbuild
from tests import layernorm_forms as forms


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return pkg.load()


def every_size():
    rng = random.Random(0)
    rows = [1, 2, 9, 130, 152, 200, 700, 2500, 9000, 60000, 250000, (1 << 31) - 1]
    for d in [*range(1, 300), *range(2020, 2060), *range(4070, 4110), *range(6120, 6160), *range(8160, 8210), 16384, 16392, 32768,
              32776, 1 << 24, *(rng.randint(1, 40000) for _ in range(300))]:
        yield from ((r, d) for r in rows)


@pytest.mark.parametrize("sms", [152, 148, 160])
@pytest.mark.parametrize("part,sizes", [(0, forms.FORWARD), (1, forms.BACKWARD)])
def test_the_tests_sizes_reach_every_kernel(part, sizes, sms):
    assert forms.kinds(part, sizes, sms) == forms.kinds(part, every_size(), sms)


@pytest.mark.parametrize("sms", [152, 148, 160])
def test_the_tests_sizes_begin_inside_a_vector(sms):
    for rows, d in forms.STRADDLE:
        assert pkg.tfl_selftest_layernorm_plan(d, pkg.TFL_F32, 1, rows, True, sms) == (pkg.TFL_LN_FORM_STRADDLE, 512, 1), (rows, d)


@pytest.mark.parametrize("sms", [1, 152])
def test_every_plan_is_within_the_kernels_limits(sms):
    for rows, d in every_size():
        for res in (pkg.TFL_F32, pkg.TFL_F16):
            for part in (0, 1):
                form, threads, vectors = pkg.tfl_selftest_layernorm_plan(d, res, part, rows, True, sms)
                loose = pkg.tfl_selftest_layernorm_plan(d, res, part, rows, False, sms)
                assert loose == (pkg.TFL_LN_FORM_VALUES if d <= 8192 else pkg.TFL_LN_FORM_ANY, 0, 0)
                if form >= pkg.TFL_LN_FORM_VALUES:
                    assert (threads, vectors) == (0, 0) and (form == pkg.TFL_LN_FORM_VALUES) == (d <= 8192)
                    continue
                inside = form == pkg.TFL_LN_FORM_STRADDLE
                assert inside == (d % 8 != 0) and threads % 32 == 0 and threads <= (1024 if part == 0 else 512)
                assert threads * vectors * 8 >= d + (14 if inside else 0)  # wherever in a vector the row begins


@pytest.mark.parametrize("sms", [152, 600])
def test_rows_that_begin_inside_a_vector_take_wide_blocks_backward(sms):
    """Their kernels of 384 and 512 threads are the only ones there are."""
    for rows, d in [*every_size(), (133334, 15), (64516, 31), (31747, 63), (15749, 127), (7844, 255)]:
        form, threads, vectors = pkg.tfl_selftest_layernorm_plan(d, pkg.TFL_F32, 1, rows, True, sms)
        if form == pkg.TFL_LN_FORM_STRADDLE:
            assert (threads, vectors) in ((512, 1), (384, 2), (512, 2)), (rows, d)


@pytest.mark.parametrize("args", [(0, 0, 0, 1, 1, 152), ((1 << 24) + 1, 0, 0, 1, 1, 152), (64, 3, 0, 1, 1, 152), (64, 4, 0, 1, 1, 152),
                                  (64, 0, -1, 1, 1, 152), (64, 0, 2, 1, 1, 152), (64, 0, 0, 0, 1, 152),
                                  (64, 0, 0, 1 << 31, 1, 152), (64, 0, 0, 1, 1, -1)])
def test_refusals(args):
    with pytest.raises(pkg.TflError) as e:
        pkg.tfl_selftest_layernorm_plan(*args)
    assert e.value.code == pkg.TFL_ERR_INVALID_ARG and str(e.value)
