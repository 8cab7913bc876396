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
