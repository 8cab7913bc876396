"""Where the kernels that may start early wait for the kernels in front of them, read body by body from the sources
(CPU).  Only `griddepcontrol.wait` makes what earlier kernels wrote visible to a kernel that was let in early, so each
executes it once, whatever its arguments are, and reads nothing of theirs before.  (The two fused kernels of the
forward bring biases in before it: parameters that were packed when the handle was made.)"""
import glob
import os
import re

import pytest

from tests.test_ops_sources import CSRC, _code

FILES = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu*")))
READS = (r"\b(load8|load1|load_raw|load_first|load_once|load_params2|load_cols|load_gamma|widen)\s*[<(]|\btma_load|\bbulk_load|"
         r"__ld\w+\(|\*\s*reinterpret_cast<const|\b(a|args)\.\w+\[|\bld\.global")


PACKED = ("postchain.cu", "stack.cu")


def closing(code, at):
    """The index behind the brace that closes the one at `at`."""
    depth = 0
    for i in range(at, len(code)):
        depth += (code[i] == "{") - (code[i] == "}")
        if depth == 0:
            return i + 1
    raise AssertionError("unbalanced braces")


def bodies(code):
    """(name, body between its braces) of each kernel of a source without comments."""
    for at in re.finditer(r"__global__ void", code):
        head = code[at.end():code.index("{", at.end())]
        name = [n for n in re.findall(r"(\w+)\s*\(", head) if n not in ("__launch_bounds__", "__attribute__", "tile_threads")][0]
        start = at.end() + len(head)
        yield name, code[start + 1:closing(code, start) - 1]


def without_lambdas(body):
    """The body without its named lambdas, and their names."""
    names = []
    while True:
        at = re.search(r"\bauto (\w+) = \[[^\]]*\]\([^)]*\)( -> \w+)? \{", body)
        if not at:
            return body, names
        names.append(at.group(1))
        body = body[:at.start()] + body[closing(body, at.end() - 1):]


def problem(body, packed=False):
    """What is wrong with a kernel that lets the next one start early; None if nothing is."""
    body, lambdas = without_lambdas(body)
    waits = [m.start() for m in re.finditer(r"\bgrid_wait_prior\(\)", body)]
    if len(waits) != 1:
        return "%d waits" % len(waits)
    before = body[:waits[0]]
    if before.count("{") != before.count("}"):
        return "a wait inside a block"
    if before.rstrip()[-1:] not in (";", "{", "}"):
        return "a conditional wait"
    if not packed and re.search(READS, before):
        return "a read before the wait"
    if any(re.search(r"\b%s\(" % name, before) for name in lambdas):
        return "a lambda called before the wait"
    return None


@pytest.mark.parametrize("name", FILES)
def test_every_kernel_that_starts_early_waits_before_it_reads(name):
    code = _code(os.path.join(CSRC, name))
    for kernel, body in bodies(code):
        if "grid_launch_dependents" in body or "grid_wait_prior" in body:
            wrong = problem(body, name in PACKED)
            assert wrong is None, (kernel, wrong)


def test_every_kernel_launched_to_start_early_is_looked_at():
    """The names launch_dependent and the tiled kernel's own launch are given, against the bodies that wait."""
    launched, waiting = set(), set()
    for name in FILES + ["kernels.h"]:
        code = _code(os.path.join(CSRC, name))
        launched |= set(re.findall(r"\blaunch_dependent\(\s*(\w+)", code))
        launched |= set(re.findall(r"cudaLaunchKernelEx\(&cfg, (\w+)<", code))
        waiting |= {kernel for kernel, body in bodies(code) if "grid_wait_prior();" in body}
    launched -= {"void", "kern"}
    assert len(launched) >= 20 and launched <= waiting, launched - waiting


def test_the_two_instructions_stand_in_two_functions_only():
    seen = 0
    for name in FILES + ["host.h", "kernels.h", "ops.h"]:
        code = _code(os.path.join(CSRC, name))
        seen += code.count("griddepcontrol")
        assert name == "ptx.cuh" or "griddepcontrol" not in code, name
    code = _code(os.path.join(CSRC, "ptx.cuh"))
    assert seen == 2
    # neither under another name
    assert len(re.findall(r"\bgrid_wait_prior\(\)", code)) == 1 and len(re.findall(r"\bgrid_launch_dependents\(\)", code)) == 1


@pytest.mark.parametrize("body,wrong", [
    ("grid_launch_dependents(); grid_wait_prior(); float v = a.x[0];", None),
    ("grid_launch_dependents(); float v = a.x[0]; grid_wait_prior();", "a read before the wait"),
    ("grid_launch_dependents(); if (link) grid_wait_prior(); float v = a.x[0];", "a conditional wait"),
    ("grid_launch_dependents(); if (link) { grid_wait_prior(); }", "a wait inside a block"),
    ("grid_launch_dependents(); float v = a.x[0];", "0 waits"),
    ("auto get = [&](int i) { return a.x[i]; }; grid_wait_prior(); get(0);", None),
    ("auto get = [&](int i) { return a.x[i]; }; get(0); grid_wait_prior();", "a lambda called before the wait")])
def test_the_rule_sees_each_mistake(body, wrong):
    assert problem(body) == wrong
