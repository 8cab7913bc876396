"""Sizes that take the gated feed-forward through every form of its kernels, in every mode."""
import attention_qkv_gemm_gb300 as pkg

# tokens, d_model, d_ff: sizes that no tile divides, several k-blocks a tile, for lone CTAs and pairs
# more tiles than run at once; rows of whole 128-byte lines in the last two
FORWARD = [(9, 1000, 136), (274, 136, 6496), (17, 472, 144), (7824, 216, 304), (6763, 136, 584), (2600, 1024, 2056),
           (1001, 320, 4104)]
E4M3 = [(5, 1040, 144), (261, 288, 6960), (17, 1232, 144), (6697, 528, 288), (429, 272, 8544), (2600, 1024, 2064),
        (1001, 640, 4112)]
BACKWARD = [(143, 136, 4960), (131, 1048, 3216), (498, 136, 136), (137, 712, 4904), (7531, 392, 136), (6845, 600, 136),
            (18, 136, 208), (3094, 2512, 136), (274, 136, 6496), (17, 472, 144), (7824, 216, 304), (6763, 136, 584),
            (2600, 1024, 2048), (1001, 320, 4104)]

TILED = (pkg.TFL_GLU_FORM_LONE, pkg.TFL_GLU_FORM_SHARED, pkg.TFL_GLU_FORM_PAIR, pkg.TFL_GLU_FORM_WIDE)


def reached(units=None):
    """(part, e4m3, form) of every launch of these sizes; units as tfl_selftest_glu_plan takes them."""
    got = set()
    for sizes, kind, parts in ((FORWARD, pkg.TFL_BF16, (0,)), (E4M3, pkg.TFL_E4M3, (0,)), (BACKWARD, pkg.TFL_BF16, (1, 2, 3))):
        for tokens, d, f in sizes:
            for part in parts:
                form = pkg.tfl_selftest_glu_plan(d, f, kind, part, tokens, units)[0]
                got.add((part, kind == pkg.TFL_E4M3, form))
    return got


WANTED = ({(0, f8, form) for f8 in (False, True) for form in (pkg.TFL_GLU_FORM_FEW, *TILED)} |
          {(part, False, form) for part in (1, 2, 3) for form in TILED})
