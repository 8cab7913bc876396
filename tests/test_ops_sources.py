"""Rules that the kernels' sources keep, read from the files themselves (CPU)."""
import glob
import os
import re

import attention_qkv_gemm_gb300 as pkg

CSRC = os.path.join(os.path.dirname(os.path.abspath(pkg.__file__)), "csrc")


def _code(path):
    """A source's text without comments, its string literals joined where they are adjacent."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    return re.sub(r'"\s*"', "", text)


def test_no_copy_is_multicast():
    """Each CTA issues its own copies: the library is loaded by every rank of a replicated run, and a
    buffer may be another GPU's.  (A commit may arrive on the barriers of several CTAs.)"""
    files = glob.glob(os.path.join(CSRC, "*.cu*"))
    assert len(files) > 10
    for path in files:
        for line in re.findall(r'"[^"]*multicast[^"]*"', _code(path)):
            assert line.startswith('"tcgen05.commit.'), (os.path.basename(path), line)


def test_only_what_no_kernel_writes_is_read_through_the_non_coherent_path():
    """A kernel of these may be resident before the one in front of it has written x or its scales,
    and `ld.global.nc` is defined only for data that nobody writes meanwhile: weights, their scales
    and gamma."""
    ours = r"(args|a)\.(g_scale|u_scale|gamma) \+|reinterpret_cast<const float4\*>\(p\)"  # p: load_gamma's
    seen = 0
    for name in ("glu.cu", "glu_few.cu", "rmsnorm.cu"):
        code = _code(os.path.join(CSRC, name))
        for at in re.finditer(r"__ldg\((.{60})", code, re.S):
            assert re.match(ours, at.group(1)), (name, at.group(1))
            seen += 1
        assert len(re.findall(r"\.nc\b", code)) == (name == "glu_few.cu"), name  # load_once
        for at in re.finditer(r"load_once\((?!const)(\w+)", code):
            assert at.group(1) in ("wg", "wu"), (name, at.group(1))
            seen += 1
    assert seen >= 8
