"""Sizes that take the linear layer through every form of its kernels, in every part."""
import attention_qkv_gemm_gb300 as pkg

# tokens, d_in, d_out: sizes that no tile divides, several k-blocks a tile, for lone CTAs and pairs more
# tiles than run at once; rows of whole 128-byte lines in the last two
FORWARD = [(16, 184, 40), (7082, 192, 144), (19, 456, 40), (5876, 136, 1312), (6761, 144, 1200), (2600, 1024, 2056),
           (1001, 320, 4104)]
E4M3 = [(16, 320, 80), (7270, 384, 160), (17, 1024, 80), (2951, 272, 2576), (5860, 272, 1472), (2600, 1024, 2064),
        (1001, 640, 4112)]
DX = [(6557, 264, 152), (23, 40, 488), (7768, 608, 200), (6550, 1192, 136), (2600, 1024, 2056), (1001, 320, 4104)]
DW = [(151, 704, 2560), (460, 48, 48), (194, 2528, 2232), (136, 3280, 2592), (2600, 1024, 2056), (1001, 320, 4104)]

# few outputs and many tokens: dw over shares of the tokens
SHARES = [(41798, 120, 224), (50001, 128, 384), (30011, 8, 8), (20000, 64, 72), (49881, 1160, 176), (30011, 264, 520),
          (40000, 512, 520), (60001, 1024, 264)]

TILED = (pkg.TFL_GLU_FORM_LONE, pkg.TFL_GLU_FORM_SHARED, pkg.TFL_GLU_FORM_PAIR, pkg.TFL_GLU_FORM_WIDE)


def reached(units=None):
    """(part, e4m3, form) of every launch of these sizes; units as tfl_selftest_linear_plan takes them."""
    got = set()
    for sizes, kind, part in ((FORWARD, pkg.TFL_BF16, 0), (E4M3, pkg.TFL_E4M3, 0), (DX, pkg.TFL_BF16, 1), (DW, pkg.TFL_BF16, 2)):
        for tokens, k, n in sizes:
            got.add((part, kind == pkg.TFL_E4M3, pkg.tfl_selftest_linear_plan(k, n, kind, part, tokens, units)[0]))
    return got


WANTED = ({(0, f8, form) for f8 in (False, True) for form in (pkg.TFL_GLU_FORM_FEW, *TILED)} |
          {(part, False, form) for part in (1, 2) for form in TILED})


def dealt(units=None):
    """The forms of the SHARES sizes' dw, each of which has more tiles than its outputs."""
    got = set()
    for tokens, k, n in SHARES:
        form, columns, tiles, _ = pkg.tfl_selftest_linear_plan(k, n, pkg.TFL_BF16, 2, tokens, units)
        assert tiles > -(-n // (256 if form >= pkg.TFL_GLU_FORM_PAIR else 128)) * -(-k // columns), (tokens, k, n)
        got.add(form)
    return got


DEALT = {pkg.TFL_GLU_FORM_LONE, pkg.TFL_GLU_FORM_PAIR}
