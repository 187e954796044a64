"""GPU tests of the page operations in the sizes of a whole model: more layers, entries and copies than
one launch takes (8 layers, 512 pieces of 2,048 bytes or runs of 128 table entries)."""
import random

import numpy as np
import pytest
import torch

from tests.attend_helpers import BS, compact_ref, pages_of
from tests.test_gpu_pages import Pool, _tq

pytestmark = pytest.mark.gpu


class Model(Pool):
    """A pool with the given (H_kv, slot stride) a layer; every third layer lies between two others."""

    def __init__(self, batch, cols, pool, shapes, seed=0, reserve=()):
        super().__init__(batch, cols, pool, layers=0, seed=seed, reserve=reserve)
        g = torch.Generator("cuda").manual_seed(seed)
        for i, (h, s) in enumerate(shapes):
            size = (pool, 3, BS, h, s) if i % 3 == 1 else (pool, BS, h, s)
            x = torch.randint(0, 256, size, dtype=torch.uint8, device="cuda", generator=g)
            self.pages.append(x[:, 1] if i % 3 == 1 else x)
            self.np_pages.append(self.pages[-1].cpu().numpy())


MIXED = [(1, 136), (2, 104), (3, 88), (8, 136), (1, 8), (2, 136), (5, 40), (4, 104), (1, 264)]
WIDE = [(2, 136), (1, 16), (4, 104), (8, 136)]            # rows of 16-byte multiples only


@pytest.mark.parametrize("shapes", [MIXED, MIXED * 3 + WIDE, WIDE * 32], ids=["9", "31", "128"])
def test_every_layer_is_copied(shapes):
    """Forks of partly filled pages, then copy on write in most rows, in 9 and more layers."""
    tq = _tq()
    p = Model(12, 6, 70, shapes, reserve=[2, 9])
    p.resize(tq, [40, 17, 32, 1, 0, 0, 0, 0, 0, 0, 0, 0])
    p.fork(tq, [0, 0, 1, 2, 3, 0, 1, 5], [4, 5, 6, 7, 8, 9, 10, 11])
    # cut into shared pages, then grow: copy on write
    p.resize(tq, [20, 17, 20, 1, 40, 5, 17, 30, 1, 31, 3, 0])
    p.resize(tq, [21, 33, 40, 2, 41, 6, 18, 31, 0, 96, 16, 7])
    p.fork(tq, [9], [8])
    p.resize(tq, [96] * 12, window=20, sinks=3)           # 72 entries of 68 pages, 4 and more of them shared
    p.resize(tq, [0] * 12)
    assert tq.get_device_error() == 0
    assert p.refs.sum() == 2


def test_refusals_in_two_launches():
    tq = _tq()
    p = Model(6, 6, 20, MIXED, reserve=[0, 19])
    p.resize(tq, [40, 17, 60, 0, 0, 0])                   # 9 of 18 pages
    p.resize(tq, [41, 96, 96, 70, 1, 97])                 # 1: 4 more, 2: 2, 3: 5 with 3 left; 4 after it; a bad length
    assert tq.get_device_error() == tq.DEVERR_NO_PAGES | tq.DEVERR_SEQLEN_RANGE
    p.fork(tq, [0, 1, 0, 9, 0], [3, 4, 5, 5, 1])          # two copies; an index, a child named twice or in use
    assert tq.get_device_error() == tq.DEVERR_SEQ_INDEX
    p.resize(tq, [0] * 6)
    assert p.refs.sum() == 2


def test_many_copies_in_few_layers():
    """700 children with a partly filled page each, in two layers: too many pieces for one launch."""
    tq = _tq()
    n = 700
    p = Model(n + 8, 5, 3 * n, [(2, 104), (8, 136)])
    p.resize(tq, [70, 1, 33, 16, 5, 79, 64, 18] + [0] * n)
    p.fork(tq, [i % 8 for i in range(n)], list(range(8, n + 8)))
    p.resize(tq, [int(x) - int(x) % 7 for x in p.lens])
    p.resize(tq, [min(80, int(x) + 1 + i % 3) for i, x in enumerate(p.lens)])
    assert np.any(p.lens[8:] % BS)
    p.resize(tq, [0] * (n + 8))
    assert tq.get_device_error() == 0
    assert p.refs.sum() == 0


@pytest.mark.parametrize("shapes", [[(1, 8)], [(1, 8)] * 9], ids=["1", "9"])
def test_long_rows(shapes):
    """Rows of over 1,024 entries (a block's share of a fork, four turns of a release's threads)."""
    tq = _tq()
    cols = 2300
    p = Model(5, cols, 6000, shapes)
    p.resize(tq, [2200 * BS - 3, 1024 * BS, 1025 * BS + 1, 0, 0])
    p.fork(tq, [0, 2], [3, 4])
    p.resize(tq, [2200 * BS - 2, 1030 * BS, 7, 1100 * BS, 1026 * BS], window=1100 * BS, sinks=40)
    p.resize(tq, [3, 0, 7, 0, 1])
    p.resize(tq, [0] * 5)
    assert tq.get_device_error() == 0
    assert p.refs.sum() == 0


@pytest.mark.parametrize("shapes", [MIXED, WIDE, WIDE * 3, MIXED * 14 + WIDE[:2]], ids=["9", "4w", "12w", "128"])
def test_compact_in_every_layer(shapes):
    tq = _tq()
    rng = np.random.default_rng(len(shapes))
    batch, length, keep = 3, 90, 41
    p = Model(2 * batch, 8, 60, shapes)
    p.resize(tq, [length] * batch + [keep] * batch)
    counts = np.asarray([keep, 16, 0], np.int32)
    pos = np.stack([rng.permutation(length)[:keep] for _ in range(batch)]).astype(np.int32)
    t, l, _ = p.dev
    tq.pages_compact(p.pages, t[:batch], l[:batch], p.i32(pos), p.i32(counts), t[batch:])
    compact_ref(p.np_pages, p.table[:batch], p.lens[:batch], pos, counts, p.table[batch:])
    p.same(p.i32([[0, 0]]), np.zeros((1, 2), np.int32))
    assert tq.get_device_error() == 0


@pytest.mark.parametrize("layers", [1, 9])
def test_random_runs_in_two_launches(layers):
    tq = _tq()
    rng = random.Random(layers)
    batch, cols, pool = 130, 1100, 40000
    p = Model(batch, cols, pool, [(1, 8), (1, 24), (2, 8)][:layers] if layers < 3 else [(1, 8), (1, 24), (2, 8)] * 3,
              reserve=rng.sample(range(pool), 4000))
    for _ in range(6):
        new = [rng.choice((int(n), rng.randrange(cols * BS + 1), min(cols * BS, int(n) + 1), 0, 0)) for n in p.lens]
        p.resize(tq, new, window=rng.choice((0, 500)), sinks=rng.choice((0, 17)))
        empty = [b for b in range(batch) if p.lens[b] == 0]
        children = rng.sample(empty, len(empty) // 2)
        if children:
            p.fork(tq, [rng.randrange(batch) for _ in children], children)
    assert tq.get_device_error() in (0, tq.DEVERR_NO_PAGES)
    assert pages_of(int(p.lens.max())) > 1024


def test_the_widest_table():
    """2^26 - 1 columns: a fork's grid ends below what a launch takes, and it loops."""
    tq = _tq()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")     # noqa: E731
    cols, pool = (1 << 26) - 1, 40_000
    table = torch.full((2, cols), -1, dtype=torch.int32, device="cuda")
    pages = torch.zeros(pool, BS, 1, 8, dtype=torch.uint8, device="cuda")
    lens, refs, moves = i32([0, 0]), torch.zeros(pool, dtype=torch.int32, device="cuda"), i32([[9, 9]] * 2)
    n = 33_000 * BS + 5                                     # 33,001 pages
    tq.pages_resize(pages, table, lens, i32([n, 0]), refs, moves)
    pages[33_000] = 7
    tq.pages_fork(pages, table, lens, refs, i32([0]), i32([1]), moves[:1])
    assert lens.tolist() == [n, n] and moves[0].tolist() == [33_000, 33_001]
    assert torch.equal(table[0, :33_001], torch.arange(33_001, dtype=torch.int32, device="cuda"))
    assert torch.equal(table[1, :33_000], table[0, :33_000]) and int(table[1, 33_000]) == 33_001
    assert torch.all(refs[:33_000] == 2) and refs[33_000:33_002].tolist() == [1, 1] and not refs[33_002:].any()
    assert torch.equal(pages[33_001], pages[33_000])
    # the last entry of a row counts as any other
    lens.copy_(i32([0, cols * BS]))
    table[1, cols - 1] = 39_000
    refs[39_000] = 1
    tq.pages_resize(pages, table, lens, i32([0, 16]), refs, moves)
    assert int(refs[39_000]) == 0 and int(table[1, cols - 1]) == -1 and lens.tolist() == [0, 16]
    assert tq.get_device_error() == 0
