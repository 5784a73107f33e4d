"""How mixllm_kv8_append shares a list of slots among its warps, as a model: every
tile of 16 places finds the runs that begin in it from the 32 places from its
first one on and the last token before them, and what lies too far behind its
block's first token from the 32 places before.  Checked against what the header says of whole lists: a block is one
run's, whatever is skipped inside it, and what is left out is recorded (CPU only)."""
import random

import pytest

BLOCK, WINDOW = 16, 32


def _kernel(slots):
    """(runs, recorded): runs as lists of places; the kernel's steps, lane by lane."""
    runs, recorded = [], False
    T = len(slots)
    at = lambda t: slots[t] if 0 <= t < T else -1  # noqa: E731
    for t0 in range(0, T, BLOCK):
        slot = [at(t0 + i) for i in range(WINDOW)]
        back = [at(t0 + i - WINDOW) for i in range(WINDOW)]
        there = [i for i in range(WINDOW) if slot[i] >= 0]
        behind = [i for i in range(WINDOW) if back[i] >= 0]
        last = back[behind[-1]] if behind else -1
        if not behind and any(i < BLOCK for i in there):
            last = next((slots[t] for t in range(t0 - WINDOW - 1, -1, -1) if slots[t] >= 0), -1)
        begin = []
        for n, i in enumerate(there):
            prev = slot[there[n - 1]] if n else last
            if prev < 0 or prev // BLOCK != slot[i] // BLOCK:
                begin.append(i)
        own = [i for i in there if i < BLOCK]
        if own:  # the tile's first block: does it go on from before, and too far?
            block = slot[own[0]] // BLOCK
            far = next((own[n - 1] for n in range(1, len(own)) if slot[own[n]] // BLOCK != block), own[-1])
            same = [i for i in behind if back[i] // BLOCK == block]
            other = [i for i in behind if i not in same]
            chain = [i for i in same if not other or i > other[-1]]
            recorded |= far + WINDOW - chain[0] >= BLOCK if chain else not behind and last >= 0 and last // BLOCK == block
        for first in (i for i in begin if i < BLOCK):
            later = [i for i in begin if i > first]
            rest = [i for i in there if i >= first and (not later or i < later[0])]
            run = [i for i in rest if i < first + BLOCK]
            recorded |= rest != run
            runs.append([t0 + i for i in run])
    return runs, recorded


def _header(slots):
    """The same from the definition: tokens of a block that follow one another, within 16 places of the first."""
    runs, recorded, block, first = [], False, -1, 0
    for t, slot in enumerate(slots):
        if slot < 0:
            continue
        if slot // BLOCK != block:
            block, first = slot // BLOCK, t
            runs.append([])
        if t - first < BLOCK:
            runs[-1].append(t)
        else:
            recorded = True
    return runs, recorded


@pytest.mark.parametrize("slots", [
    [0, 1, -1, 2], [-1, 0, -1, -1, 1, 16, -1, 17], [14, 15, -1, 16], [0] + 14 * [-1] + [1], [0] + 15 * [-1] + [1],
    [0] + 40 * [-1] + [1], [0] + 200 * [-1] + [1], [0] + 300 * [-1] + [16], 60 * [-1] + [3, 4], list(range(5, 70)),
    [0] * 40, [5, -1, 6] + 29 * [-1] + [7], [t if t % 3 else -1 for t in range(100)]], ids=str)
def test_chosen_lists(slots):
    assert _kernel(slots) == _header(slots)


def _list(rng):
    """Requests' tokens in blocks of their own, with places left out inside and runs of padding between."""
    out, block = [], 0
    for _ in range(rng.randrange(1, 8)):
        first, n = rng.randrange(BLOCK), rng.choice([1, 2, 5, 16, 40, 90])
        for t in range(first, first + n):
            out.append(block * BLOCK + t)
            while rng.random() < rng.choice([0, 0, 0.1, 0.7]):
                out.append(-1)
        if rng.random() < 0.3:  # some of them left out in their places
            out = [-1 if rng.random() < 0.3 else s for s in out]
        out += [-1] * rng.choice([0, 0, 1, 7, 15, 16, 17, 31, 33, 100, 200])
        block += -(-(first + n) // BLOCK) if rng.random() < 0.9 else 0  # seldom the same block once more
    return out


def test_lists_of_all_kinds():
    rng = random.Random(1)
    kept = recorded = 0
    for _ in range(1500):
        slots = _list(rng)
        got = _kernel(slots)
        assert got == _header(slots), slots
        recorded += got[1]
        kept += not got[1]
    assert kept > 200 and recorded > 200


def test_a_block_is_one_runs():
    """Where nothing is recorded, no two runs of neighbouring tokens share a block, so no two warps write one scale."""
    rng = random.Random(2)
    for _ in range(500):
        slots = _list(rng)
        runs, recorded = _kernel(slots)
        blocks = [slots[r[0]] // BLOCK for r in runs]
        assert all(slots[t] // BLOCK == b for r, b in zip(runs, blocks) for t in r)
        assert all(a != b for a, b in zip(blocks, blocks[1:]))
        if not recorded:
            assert sorted(t for r in runs for t in r) == [t for t, s in enumerate(slots) if s >= 0]
