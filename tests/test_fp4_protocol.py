"""CPU models of the barrier protocols of the kernels over a 4-bit pool.

Extend (attn_kernel, csrc/attention.cu): warp 10 copies K tiles and warp 11 V
tiles into their stages once the tensor core has released them; a tile's
landing is a phase of its stage's raw barrier, on which warps 12-13 (K) and
14-15 (V) wait before they convert in place and mark the stage full.  The
other roles are those of the model in test_barrier_protocol.py.

Decode (decode_fp4_kernel, csrc/fp4_decode.cu): the warps of a stream copy
every tile together and read their own heads' part of it; a warp refills the
stage before the one it has just read, once every warp of the stream has read
it."""
import random

import pytest

from test_barrier_protocol import RING, _Bar, _Model, _random_units


class _Fp4Extend(_Model):
    def __init__(self, units, seed, mistake=None, stages=(3, 2, 3)):
        super().__init__(units, seed, mistake, stages=stages)
        for s in range(RING):  # two warpgroups, MMA, two copying and two converting roles
            self.bars[f"UE{s}"] = _Bar(f"UE{s}", 7)
        for s in range(self.NI):
            self.bars[f"IE{s}"] = _Bar(f"IE{s}", 2)
        for pre, n in (("K", self.NK), ("V", self.NV)):
            for s in range(n):
                self.bars[f"L{pre}{s}"] = _Bar(f"L{pre}{s}", 1)

    def _roles(self):
        return {"index": self._index(), "wg0": self._softmax(0), "wg1": self._softmax(1), "mma": self._mma(),
                **{f"copy {p}": self._copy_one(p) for p in "KV"},
                **{f"convert {p}": self._convert(p) for p in "KV"}}

    def _copy_one(self, pre):
        n = self.NK if pre == "K" else self.NV
        c = ic = 0
        for op in self._units():
            if op[0] != "unit":
                yield op
                continue
            if op[1] is None:
                return
            for _ in range(op[1]["nt"]):
                si = ic % self.NI
                yield self._wait(f"IF{si}", ic // self.NI)
                yield ("arrive", f"IE{si}")
                ic += 1
                if c >= n and self.mistake != "copied before release":
                    yield self._wait(f"{pre}E{c % n}", c // n - 1)
                yield ("commit", f"L{pre}{c % n}")  # lands some time later
                c += 1

    def _convert(self, pre):
        n = self.NK if pre == "K" else self.NV
        c = 0
        for op in self._units():
            if op[0] != "unit":
                yield op
                continue
            if op[1] is None:
                return
            for _ in range(op[1]["nt"]):
                if self.mistake != "converted before landing":
                    yield self._wait(f"L{pre}{c % n}", c // n)
                yield ("use", f"L{pre}{c % n}", c // n)
                yield ("arrive", f"{pre}F{c % n}")
                c += 1


@pytest.mark.parametrize("stages", [(3, 2, 3), (5, 5, 4)])
def test_extend_protocol(stages):
    rng = random.Random(2)
    for t in range(200):
        _Fp4Extend(_random_units(rng, rng.randint(1, 12)), seed=t, stages=stages).run()


@pytest.mark.parametrize("mistake", ["copied before release", "converted before landing"])
def test_extend_model_catches_planted_mistakes(mistake):
    rng = random.Random(3)
    with pytest.raises(AssertionError):
        for t in range(200):
            _Fp4Extend(_random_units(rng, rng.randint(1, 12)), seed=t, mistake=mistake).run()


# ------------------------------------------------------------------ decode
def _decode_stream(heads, tiles, stages, rng, mistake=None):
    """Random interleaving of the stream's warps; every tile read must be the
    one its stage holds, landed from every warp, and no stage may be refilled
    while a warp still has to read it."""
    full = [0] * stages                     # arrivals of landed copies
    empty = [0] * stages
    held = [[None] * heads for _ in range(stages)]  # tile whose part warp w copied last
    readers = [set() for _ in range(stages)]        # warps that have read the stage's tile
    landing = []

    def copy(w, tile):
        s = tile % stages
        if tile >= stages:
            assert len(readers[s]) == heads or held[s][w] == tile, f"tile {tile} over an unread stage"
        landing.append((w, s, tile))

    def land(k):
        w, s, tile = landing.pop(k)
        held[s][w] = tile
        full[s] += 1
        if all(h == tile for h in held[s]):
            readers[s] = set()

    def warp(w):
        for s in range(min(stages - 1, tiles)):
            copy(w, s)
        for t in range(tiles):
            s = t % stages
            while full[s] < heads * (t // stages + 1):
                yield False
            assert all(h == t for h in held[s]), f"warp {w} reads tile {t} from {held[s]}"
            yield True
            readers[s].add(w)
            empty[s] += 1
            if t + stages - 1 < tiles:
                f = (s - 1) % stages
                if t > 0:
                    need = heads * ((t - 1) // stages + 1)
                    while empty[f] < need and mistake != "no empty wait":
                        yield False
                copy(w, t + stages - 1)
                yield True

    live = {w: warp(w) for w in range(heads)}
    idle = 0
    while live:
        if landing and rng.random() < 0.4:
            land(rng.randrange(len(landing)))
            idle = 0
        w = rng.choice(list(live))
        try:
            idle = 0 if next(live[w]) else idle + 1
        except StopIteration:
            del live[w]
        assert idle < 20000, "deadlock"


@pytest.mark.parametrize("stages", [3, 6])
def test_decode_stream_protocol(stages):
    rng = random.Random(4)
    for _ in range(150):
        _decode_stream(rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 3, 4, 9, 20]), stages, rng)


def test_decode_stream_model_catches_a_missing_wait():
    rng = random.Random(5)
    with pytest.raises(AssertionError):
        for _ in range(150):
            _decode_stream(rng.choice([2, 3, 8]), 20, 3, rng, "no empty wait")
