"""Sizes that take layer norm through every kernel, and those that begin inside a vector through every cut of the
threads into rows.  Row counts go by the dispatch's own rule on a GPU of up to 160 SMs: forward from 16 rows an SM
(one past 2034 columns), backward from 2 million values (8 million past 4082 columns)."""
import attention_qkv_gemm_gb300 as pkg

# rows, columns
FORWARD = [(300, 72), (300, 1000), (300, 1032), (300, 4096), (40, 4104), (40, 16384), (3, 32768), (3, 5), (40, 1001), (3, 8191),
           (3, 9001), (2600, 250), (2600, 2033), (2600, 2034), (200, 2035), (200, 4082), (200, 4083), (200, 8178)]
BACKWARD = [(300, 1024), (90000, 8), (2500, 2048), (300, 4096), (300, 5120), (300, 8192), (300, 16384), (3, 5), (300, 1001),
            (3, 8191), (3, 9001), (8000, 255), (1001, 4082), (2003, 4099), (1400, 6130), (1400, 6131), (1000, 8178)]

# rows that begin inside a vector, backward: 2 to 32 threads a row with several rows a warp (more than 32 groups a
# block up to 50 columns), whole warps, whole blocks; every distance of a row's start from a vector's; turns that end
# in the middle of the groups, and a group for each row
STRADDLE = [(250001, 9), (230003, 10), (200001, 12), (140001, 15), (120001, 17), (120001, 18), (70003, 31), (45001, 50), (45001, 51),
            (20000, 103), (20011, 114), (20000, 203), (10001, 242), (10001, 243), (9000, 250), (8000, 255), (8000, 257),
            (6000, 513), (6000, 516), (4001, 514), (2500, 1010), (2100, 1012), (2011, 1021), (1500, 2033), (1500, 2034)]


def kinds(part, sizes, sms=0):
    got = set()
    for rows, d in sizes:
        for res in (pkg.TFL_F32, pkg.TFL_BF16):
            got.add(kind(part, pkg.tfl_selftest_layernorm_plan(d, res, part, rows, True, sms)))
    return got


def kind(part, plan):
    """What tells one kernel from another: the forward of whole vectors takes any number of threads."""
    form, threads, vectors = plan
    return (form, 0 if part == 0 and form == pkg.TFL_LN_FORM_VECTORS else threads, vectors)
