"""Worst-case model (CPU) of one epilogue warp of the linear layer and its two shared-memory stages: a store reads its
stage until a wait says that it has, a residual's copy writes its stage from its issue to the wait on its barrier.
No stage may be written, read or copied into while either is in flight, in any epilogue and over any number of
chunks and tiles."""
import itertools

import pytest


class Hazard(Exception):
    pass


class Warp:
    def __init__(self):
        self.stores = []  # stages that committed groups may still read, oldest first
        self.flying = set()  # stages that a residual's copy may still write
        self.full = set()  # stages that hold a residual nobody has taken

    def idle(self, stage):
        if stage in self.stores or stage in self.flying:
            raise Hazard(stage)

    def stores_read(self, pending):
        while len(self.stores) > pending:
            self.stores.pop(0)

    def load(self, stage):
        self.idle(stage)
        if stage in self.full:
            raise Hazard(stage)
        self.flying.add(stage)

    def wait(self, stage):
        if stage not in self.flying:
            raise Hazard(stage)
        self.flying.remove(stage)
        self.full.add(stage)

    def write(self, stage):
        self.idle(stage)

    def store(self, stage):
        self.full.discard(stage)
        self.stores.append(stage)


def run(f32, z, res, tiles, read=lambda w, n, where: w.stores_read(n)):
    """The epilogue of `tiles`, each a number of chunks of this warp."""
    w, turn = Warp(), 0
    for chunks in tiles:
        if res and chunks:
            if z:
                turn = 0
            read(w, 1, "tile")
            w.load(turn)
        for c in range(chunks):
            for b in (0, 1):
                stage = 0 if z else turn
                more = (f32 and b == 0) or c + 1 < chunks
                if b == 0 or f32:
                    if res:
                        if not z and more:
                            read(w, 0, "ahead")
                            w.load(stage ^ 1)
                        w.wait(stage)
                    elif z and b == 1:
                        read(w, 0, "same")
                    else:
                        read(w, 1, "piece")
                w.write(stage)
                if not f32 and b == 0:
                    continue
                w.store(stage)
                turn ^= 1
                if z:
                    if b == 1:
                        read(w, 1, "z")
                        w.write(1)
                        w.store(1)
                    if res and more:
                        read(w, 0, "next")
                        w.load(0)
    if w.flying or w.full:
        raise Hazard("a residual is left over")


TILES = [t for n in (1, 2, 3) for t in itertools.product(range(4), repeat=n)]


@pytest.mark.parametrize("f32,z,res", list(itertools.product((False, True), repeat=3)))
def test_no_stage_is_touched_while_a_copy_is(f32, z, res):
    for tiles in TILES:
        run(f32, z, res, tiles)


@pytest.mark.parametrize("where,kinds", [("tile", [(False, False, True)]), ("ahead", [(False, False, True), (True, False, True)]),
                                         ("same", [(True, True, False)]), ("piece", [(False, False, False), (False, True, False)]),
                                         ("z", [(False, True, False), (False, True, True)]), ("next", [(False, True, True)])])
def test_the_model_sees_each_wait_left_out(where, kinds):
    def read(w, n, at):
        if at != where:
            w.stores_read(n)

    for kind in kinds:
        def fails(tiles):
            try:
                run(*kind, tiles, read)
            except Hazard:
                return True
            return False
        assert any(fails(t) for t in TILES), kind
