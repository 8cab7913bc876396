"""Exhaustive interleaving models of the gated feed-forward kernel's hand-offs (CPU), on the state
explorer of test_kernel_protocols.py.

csrc/glu.cu runs a CTA pair per tile: each CTA's producer fills its ring; all loads of a pair
complete on the leader's `full` barrier, which also takes the leader producer's announcement of
their bytes; the leader's issuing thread waits for it, issues the pair's products and commits to
the `empty` barriers of both CTAs; a finished accumulator is committed to both CTAs' `accf`, and
the epilogue warps of both arrive on the leader's `acce`.  Where two pairs share B, each CTA's half
of B lands in its like of the other pair as well and completes on that pair's leader, and a stage
is free for a producer only when both pairs' products have read it (an `empty` barrier counts both
commits).  A commit to several barriers is modelled as one after another, a load to several CTAs as
one load each.  The models look for deadlocks, parity waits two phases behind, and hazards: a stage
filled while a product that reads it is not complete, products issued before all they read has
landed, an accumulator read before its products or overwritten before it was read.
"""
import pytest

from tests.test_kernel_protocols import Bar, mark_pcs, run_model

STAGES = 2


def build(pairs, tiles, num_k, mutation=None):
    """Roles and barriers of one cluster of `pairs` CTA pairs (with two, one CTA stands for a pair)."""
    bars, progs, landed_on = {}, {}, {}
    ctas = 2 if pairs == 1 else 1  # modelled CTAs of a pair

    def bar(name, count):
        bars[name] = Bar(name, count)
        return name

    # arrivals of a full barrier: the announcement, A of each CTA, and B (a part from each pair's like)
    full = {(p, s): bar(f"full{p}{s}", 1 + ctas * (1 + pairs)) for p in range(pairs) for s in range(STAGES)}
    shared_empty = mutation != "own_commit_only"
    empty = {(p, c, s): bar(f"empty{p}{c}{s}", pairs if shared_empty else 1)
             for p in range(pairs) for c in range(ctas) for s in range(STAGES)}
    accf = {(p, c, a): bar(f"accf{p}{c}{a}", 1) for p in range(pairs) for c in range(ctas) for a in range(2)}
    acce = {(p, a): bar(f"acce{p}{a}", ctas if mutation != "one_epilogue_frees" else 1)
            for p in range(pairs) for a in range(2)}

    def tma(prog, on, key):
        prog.append(("tma", on, key))
        landed_on[key] = on

    for p in range(pairs):
        for c in range(ctas):
            load = []
            for j in range(tiles * num_k):
                s = j % STAGES
                load.append(("wait", empty[p, c, s], j // STAGES - 1))
                load.append(("check", "fill", (p, j)))
                if c == 0:
                    load.append(("arrive", full[p, s]))
                tma(load, full[p, s], ("A", p, c, j))
                for to in range(pairs):  # B: this CTA's part, to its like of every pair
                    tma(load, full[to, s], ("B", p, c, j, to))
            progs[f"load{p}{c}"] = load
        mma = []
        for t in range(tiles):
            a = t % 2
            mma.append(("wait", acce[p, a], t // 2 - 1))
            for kb in range(num_k):
                j = t * num_k + kb
                s = j % STAGES
                mma += [("wait", full[p, s], j // STAGES), ("check", "issue", (p, t, kb)), ("mma", f"mma{p}", ("M", p, j))]
                for q in range(pairs) if shared_empty else (p,):
                    mma += [("commit", f"mma{p}", empty[q, c, s]) for c in range(ctas)]
            mma += [("commit", f"mma{p}", accf[p, c, a]) for c in range(ctas)]
        progs[f"mma{p}"] = mma
        for c in range(ctas):
            epi = []
            for t in range(tiles):
                epi += [("wait", accf[p, c, t % 2], t // 2), ("check", "read", (p, t)), ("mark", ("read", p, t, c)),
                        ("arrive", acce[p, t % 2])]
            progs[f"epi{p}{c}"] = epi
    return progs, bars, landed_on, ctas


def explore(pairs, tiles, num_k, mutation=None):
    progs, bars, landed_on, ctas = build(pairs, tiles, num_k, mutation)
    issuers = [f"mma{p}" for p in range(pairs)]
    pos = {}
    for r in issuers:
        entries = [a for a in progs[r] if a[0] in ("mma", "commit")]
        pos.update({a[2]: (r, k) for k, a in enumerate(entries) if a[0] == "mma"})
    marks = mark_pcs(progs)

    def done(comp, key):
        r, k = pos[key]
        return comp[r] > k

    def hazard_free(kind, arg, pcs, comp, loaded):
        if kind == "fill":  # the stage's last k-block has been read, by every pair that gets this one
            _, j = arg
            return j < STAGES or all(done(comp, ("M", q, j - STAGES)) for q in range(pairs))
        if kind == "issue":
            p, t, kb = arg
            j = t * num_k + kb
            need = [("A", p, c, j) for c in range(ctas)] + [("B", q, c, j, p) for q in range(pairs) for c in range(ctas)]
            if not all(k in loaded for k in need):
                return False
            return kb > 0 or t < 2 or all(pcs[r] >= pc for k, (r, pc) in marks.items() if k[:3] == ("read", p, t - 2))
        if kind == "read":
            p, t = arg
            return all(done(comp, ("M", p, t * num_k + kb)) for kb in range(num_k))
        raise AssertionError(kind)

    return run_model(progs, bars, landed_on, issuers, hazard_free)


@pytest.mark.parametrize("pairs,tiles,num_k", [(1, 3, 1), (1, 2, 2), (2, 1, 3), (2, 2, 1)])
def test_no_deadlock_aliasing_or_hazard(pairs, tiles, num_k):
    assert explore(pairs, tiles, num_k) > 100


@pytest.mark.parametrize("mutation,pairs,tiles,num_k", [("own_commit_only", 2, 1, 3), ("one_epilogue_frees", 1, 3, 1)])
def test_the_model_catches_a_planted_mistake(mutation, pairs, tiles, num_k):
    with pytest.raises(AssertionError):
        explore(pairs, tiles, num_k, mutation)
