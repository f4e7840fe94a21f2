"""CPU model of the index ring in extend over a 4-bit pool (attn_kernel,
csrc/attention.cu): warps 10 (K) and 11 (V) wait for a tile's row indices and
then, still holding their slot of the index ring, for the tensor core to
release the stage they copy into; they give the slot back once the copies are
issued.  The index warp refills a slot after both have.  A copier that holds a
slot while it waits must not keep the index warp from what the other one, and
through it the tensor core, needs.  The other roles are those of the models in
test_fp4_protocol.py and test_barrier_protocol.py."""
import random

import pytest

from test_barrier_protocol import _Bar, _random_units
from test_fp4_protocol import _Fp4Extend


class _IndexRing(_Fp4Extend):
    def __init__(self, units, seed, mistake=None, stages=(3, 2, 3)):
        super().__init__(units, seed, mistake, stages=stages)
        self.slot = [None] * self.NI  # number of the tile whose indices each slot holds
        if mistake == "slot freed by one copier":
            for s in range(self.NI):
                self.bars[f"IE{s}"] = _Bar(f"IE{s}", 1)

    def _index(self):
        tile = 0
        for op in super()._index():
            if op[0] == "arrive" and op[1].startswith("IF"):
                assert op[1] == f"IF{tile % self.NI}"
                self.slot[tile % self.NI] = tile
                tile += 1
            yield op

    def _copy_one(self, pre):
        n = self.NK if pre == "K" else self.NV
        c = 0
        for op in self._units():
            if op[0] != "unit":
                yield op
                continue
            if op[1] is None:
                return
            for _ in range(op[1]["nt"]):
                s = c % self.NI
                yield self._wait(f"IF{s}", c // self.NI)
                if c >= n:
                    yield self._wait(f"{pre}E{c % n}", c // n - 1)
                assert self.slot[s] == c, f"copy {pre}: slot {s} holds tile {self.slot[s]}, not {c}"
                if self.mistake == "slot held for the next one" and c + 1 < sum(u["nt"] for u in self.units):
                    yield self._wait(f"IF{(c + 1) % self.NI}", (c + 1) // self.NI)
                if not (pre == "V" and self.mistake == "slot freed by one copier"):
                    yield ("arrive", f"IE{s}")
                yield ("commit", f"L{pre}{c % n}")  # lands some time later
                c += 1


# the stages of 128 and of 64 dims, and an index ring of a single slot
@pytest.mark.parametrize("stages", [(3, 2, 3), (5, 5, 4), (3, 2, 1), (5, 5, 1)])
def test_index_ring(stages):
    rng = random.Random(6)
    for t in range(200):
        _IndexRing(_random_units(rng, rng.randint(1, 12)), seed=t, stages=stages).run()


def test_model_catches_a_slot_freed_by_one_copier():
    rng = random.Random(7)
    with pytest.raises(AssertionError, match="holds tile"):
        for t in range(200):
            _IndexRing(_random_units(rng, rng.randint(1, 12)), seed=t, mistake="slot freed by one copier").run()


def test_model_catches_a_slot_held_for_the_next_one():
    """A copier that fetched the next tile's indices before it gave its slot
    back would wait for itself when the ring holds one slot."""
    rng = random.Random(8)
    with pytest.raises(AssertionError, match="deadlock"):
        for t in range(50):
            _IndexRing(_random_units(rng, rng.randint(1, 12)), seed=t, stages=(3, 2, 1),
                       mistake="slot held for the next one").run()
