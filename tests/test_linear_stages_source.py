"""The model of the linear layer's epilogue (test_linear_stages.py) against the epilogue itself (CPU): the waits, copies,
writes and stores of a chunk, each with the conditions it stands under, in the order of the source, are those of the
model's code."""
import ast
import inspect
import os
import re

from tests import test_linear_stages as model
from tests.test_launch_waits import closing
from tests.test_ops_sources import CSRC, _code

EVENTS = [(r"stores_read<(\d)>\(\)", "read"), (r"load_res\(([^,]+),", "load"), (r"wait_bounded\(&res_in\[(\w+)\]", "wait"),
          (r"store_stage\(&\w+, (\w+),", "store"), (r"(turn) \^= 1", "flip"), (r"(turn) = 0", "first"), (r"\b(continue);", "continue"),
          (r"\*at\(i\) = (z)\[i\]", "write"), (r"\*(?:s|at\(b \* 2 \+ i\)) = (\w+)", "write")]
NAMES = {"RES": "res", "Z": "z", "OUT32": "f32", "(EPI & kEpiRes)": "res", "EPI & kEpiZ": "z", "next >= 0": "more",
         "c * W < bno": "chunks", "&&": "and", "||": "or", "!": "not "}


def source():
    return _code(os.path.join(CSRC, "tile_gemm.cuh"))


def body_of(code, start):
    at = code.index(start)
    end = closing(code, code.index("{", at + len(start) - 1))
    return code[at + len(start):end - 1]


def condition(text):
    for a, b in sorted(NAMES.items(), key=lambda x: -len(x[0])):
        text = re.sub(r"(?<!\w)%s(?!\w)" % re.escape(a) if a[0].isalpha() else re.escape(a), b, text)
    return " ".join(text.split())


def split_if(code, at):
    """(condition, index behind it) of the `if` that starts at `at`."""
    begin = code.index("(", at)
    depth = 0
    for i in range(begin, len(code)):
        depth += (code[i] == "(") - (code[i] == ")")
        if depth == 0:
            return code[begin + 1:i], i + 1
    raise AssertionError("unbalanced parentheses")


def events_of_source(code):
    """(conditions, kind, argument) in order; conditions that the model does not know are left out."""
    found = []

    def known(text):
        c = condition(text)
        return [c] if re.fullmatch(r"(?:\W|\b(?:res|z|f32|more|chunks|b|and|or|not|0|1)\b)+", c) else []

    def walk(text, guards):
        i = 0
        while i < len(text):
            m = re.compile(r"\bif\b(?: constexpr)? \(").match(text, i)
            if m and (i == 0 or not text[i - 1].isalnum()):
                cond, j = split_if(text, i)
                walk(cond, guards)  # (a wait may be asked for its answer)
                i = branch(text, j, guards + known(cond))
                while (e := re.compile(r"\s*else\b").match(text, i)):
                    guards_else = guards + ["not (%s)" % c for c in known(cond)]
                    if (m := re.compile(r"\s*if\b(?: constexpr)? \(").match(text, e.end())):
                        cond2, j = split_if(text, e.end())
                        i = branch(text, j, guards_else + known(cond2))
                        cond, guards = cond2, guards_else
                    else:
                        i = branch(text, e.end(), guards_else)
                continue
            for pattern, kind in EVENTS:
                if (m := re.compile(pattern).match(text, i)):
                    found.append((tuple(guards), kind, m.group(1)))
                    break
            i += 1

    def branch(text, i, guards):
        while text[i].isspace():
            i += 1
        if text[i] == "{":
            end = closing(text, i)
            walk(text[i + 1:end - 1], guards)
            return end
        end = i + re.match(r"(?:[^;{]|\{[^}]*\})*;", text[i:], re.S).end()
        walk(text[i:end], guards)
        return end

    walk(code, [])
    return found


def events_of_model(statements):
    found = []

    def walk(body, guards):
        for s in body:
            if isinstance(s, ast.If):
                walk(s.body, guards + [ast.unparse(s.test)])
                walk(s.orelse, guards + ["not (%s)" % ast.unparse(s.test)])
            elif isinstance(s, ast.For):
                walk(s.body, guards)
            elif isinstance(s, ast.Expr) and isinstance(s.value, ast.Call):
                f, args = s.value.func, s.value.args
                if isinstance(f, ast.Name) and f.id == "read":
                    found.append((tuple(guards), "read", str(args[1].value)))
                else:
                    found.append((tuple(guards), f.attr, ast.unparse(args[0])))
            elif isinstance(s, ast.AugAssign):
                found.append((tuple(guards), "flip", s.target.id))
            elif isinstance(s, ast.Assign) and ast.unparse(s) == "turn = 0":
                found.append((tuple(guards), "first", "turn"))
            elif isinstance(s, ast.Continue):
                found.append((tuple(guards), "continue", "continue"))

    walk(statements, [])
    return found


def plain(events):
    """The same without what the two write differently: a stage is written by value in either width, one after the
    other, before the 16-bit form goes on to its second half, and parentheses."""
    out = []
    for guards, kind, what in events:
        guards = tuple(g.replace("(", "").replace(")", "") for g in guards)
        if kind == "write":
            what = "1" if what in ("z", "1") else "stage"
            guards = tuple(g for g in guards if "f32" not in g or "b" in g)
            if out and out[-1] == (guards, kind, what):
                continue
        if kind == "continue":
            guards = (" and ".join(guards),)
        out.append((guards, kind, what))
    return out


def parts():
    """The model's tile prologue and its chunk."""
    run = ast.parse(inspect.getsource(model.run)).body[0]
    tile = next(s for s in run.body if isinstance(s, ast.For))
    return [s for s in tile.body if isinstance(s, ast.If)], [s for s in tile.body if isinstance(s, ast.For)]


def chunk_source():
    return body_of(source(), "auto lin_chunk = [&](int c) -> bool {")


def check_chunk(code):
    got = [e for e in plain(events_of_source(code)) if e[1] != "first"]
    return got, plain(events_of_model(parts()[1]))


def test_a_chunk_waits_copies_and_stores_as_the_model_does():
    got, want = check_chunk(chunk_source())
    assert got == want and len(want) >= 14


def test_a_tile_begins_as_the_model_does():
    code = source()
    at = code.index("int c = part + split * half;")
    code = code[at:code.index("while ((c += H * split)", at)]
    got = plain(events_of_source(code[:code.index("const int size")] + "}"))
    assert got == plain(events_of_model(parts()[0])) and len(got) == 3


def test_nothing_is_left_in_flight_at_the_end():
    code = source()
    end = code[code.index("if (dead) break;"):code.index("if (*abort_flag)")]
    assert re.search(r"if \(res_flying & \(1u << s\)\) wait_bounded\(&res_in\[s\], \(res_phase >> s\) & 1u, dc\);\s*stores_read<0>\(\);", end)
    assert code.count("stores_read<") == 7 and code.count("load_res(") == 3 and code.count("store_stage(&") == 2


def test_every_wait_left_out_or_moved_shows():
    code = chunk_source()
    for m in re.finditer(r"stores_read<(\d)>\(\);", code):
        for other in ("", "stores_read<%d>();" % (1 - int(m.group(1)))):
            got, want = check_chunk(code[:m.start()] + other + code[m.end():])
            assert got != want, m.start()
    for a, b in (("RES && next >= 0", "next >= 0"), ("!Z && next >= 0", "next >= 0"), ("stage ^ 1, next", "stage, next"),
                 ("Z && b == 1", "Z"), ("store_stage(&tmB1, 1,", "store_stage(&tmB1, 0,")):
        assert code.count(a) == 1, a
        got, want = check_chunk(code.replace(a, b))
        assert got != want, a
