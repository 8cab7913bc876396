"""Exhaustive model (CPU) of the linear layer's backward as a chain of launches that start early: a kernel's blocks
may start once all blocks of the kernel in front of it have allowed it (or are done), a wait lasts until that kernel
is done.  LINK_FIRST waits before it allows the next one, LINK_LATER works without a wait and waits at its end."""
import pytest

PLAIN = ("allow", "wait", "work")
FIRST = ("wait", "allow", "work")
LATER = ("allow", "work", "wait")

# name, program, kernels that have to be done before its work
SLOPES = ("slopes", PLAIN, ("before",))
NEXT = ("next", PLAIN, "all")  # the next call's slopes write what every kernel of this one reads


def chain(dx, dw, shares, db, link_first=FIRST, link_later=LATER, link_db=LATER):
    ks = [("before", PLAIN, ()), SLOPES]
    if dx:
        ks.append(("dx", link_first, ("slopes",)))
    if dw:
        ks.append(("dw", link_later if dx else link_first, ("slopes",)))
    if dw and shares:
        ks.append(("sums", PLAIN, ("dw",)))
    if db:
        ks.append(("db", link_db if dx or dw else PLAIN, ("slopes",)))
    return ks + [NEXT]


def faults(kernels, blocks=2):
    """What can go wrong over all interleavings: work before what it needs, or no way on."""
    names = [k[0] for k in kernels]
    found = set()
    start = tuple((0,) * blocks for _ in kernels)  # steps done of each block; the first step means it has started
    seen, todo = {start}, [start]
    done = lambda s, k: all(p == 3 for p in s[k])
    allowed = lambda s, k: all("allow" in kernels[k][1][:p] for p in s[k])
    while todo:
        s = todo.pop()
        moved = False
        for k, (name, program, needs) in enumerate(kernels):
            if k and not allowed(s, k - 1):
                continue
            for b in range(blocks):
                p = s[k][b]
                if p == 3 or (program[p] == "wait" and k and not done(s, k - 1)):
                    continue
                if program[p] == "work":
                    for n in names[:k] if needs == "all" else needs:
                        if not done(s, names.index(n)):
                            found.add((name, n))
                moved = True
                row = s[k][:b] + (p + 1,) + s[k][b + 1:]
                t = s[:k] + (tuple(sorted(row)),) + s[k + 1:]  # blocks of a kernel are alike
                if t not in seen:
                    seen.add(t)
                    todo.append(t)
        if not moved and not done(s, len(kernels) - 1):
            found.add("stuck")
    return found


CALLS = [(dx, dw, shares, db) for dx in (0, 1) for dw in (0, 1) for shares in (0, 1) for db in (0, 1)
         if (dx or dw or db) and not (shares and not dw)]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("blocks", [1, 2])
def test_no_kernel_works_before_what_it_needs(call, blocks):
    assert faults(chain(*call), blocks) == set()


def test_the_model_sees_a_first_that_allows_before_it_waits():
    assert ("dw", "slopes") in faults(chain(1, 1, 0, 0, link_first=PLAIN))
    assert ("db", "slopes") in faults(chain(0, 1, 0, 1, link_first=PLAIN))


def test_the_model_sees_a_later_that_never_waits():
    assert ("next", "dx") in faults(chain(1, 1, 0, 0, link_later=("allow", "work", "work")))
    assert ("next", "dw") in faults(chain(0, 1, 0, 1, link_db=("allow", "work", "work")))


def test_the_model_sees_the_sum_of_shares_linked():
    ks = [("sums", LATER, k[2]) if k[0] == "sums" else k for k in chain(1, 1, 1, 0)]
    assert ("sums", "dw") in faults(ks)
