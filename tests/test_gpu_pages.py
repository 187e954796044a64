"""GPU tests of the page operations: whole state (tables, lengths, counts, moves, every byte of
every layer's pages) against a request-by-request form, and a run of the operators together."""
import random

import numpy as np
import pytest
import torch

from kv_cache_vector_append_b200 import workloads as W
from tests.attend_helpers import (BS, attend_ref, check_rows, compact_ref, fork_ref, out_eps, pages_of, resize_ref)
from tests.gpu_helpers import require_gpu, to_np_f64

pytestmark = pytest.mark.gpu


def _tq():
    require_gpu()
    import kv_cache_vector_append_b200 as tq
    return tq


class Pool:
    """Device state and its numpy twin."""

    def __init__(self, batch, cols, pool, layers=2, seed=0, reserve=()):
        g = torch.Generator().manual_seed(seed)
        shapes = [(1, 136), (2, 104), (3, 88)]
        self.np_pages, self.pages = [], []
        for i in range(layers):
            h, s = shapes[i % 3]
            if i == 1:                      # a layer that interleaves with others in one tensor
                wide = torch.randint(0, 256, (pool, 2, BS, h, s), dtype=torch.uint8, generator=g).cuda()
                self.pages.append(wide[:, 1])
            else:
                self.pages.append(torch.randint(0, 256, (pool, BS, h, s), dtype=torch.uint8, generator=g).cuda())
            self.np_pages.append(self.pages[-1].cpu().numpy())
        self.table = np.full((batch, cols), -1, np.int32)
        self.lens = np.zeros(batch, np.int32)
        self.refs = np.zeros(pool, np.int32)
        self.refs[list(reserve)] = 1
        self.dev = [torch.from_numpy(x.copy()).cuda() for x in (self.table, self.lens, self.refs)]

    def i32(self, x):
        return torch.from_numpy(np.asarray(x, np.int32).copy()).cuda()

    def resize(self, tq, new, window=0, sinks=0):
        t, l, r = self.dev
        moves = torch.full((len(self.lens), 2), 9, dtype=torch.int32, device="cuda")
        tq.pages_resize(self.pages, t, l, self.i32(new), r, moves, window=window, sinks=sinks)
        want = resize_ref(self.np_pages, self.table, self.lens, np.asarray(new), self.refs, window, sinks)
        self.same(moves, want)

    def fork(self, tq, parents, children):
        t, l, r = self.dev
        moves = torch.full((len(parents), 2), 9, dtype=torch.int32, device="cuda")
        tq.pages_fork(self.pages, t, l, r, self.i32(parents), self.i32(children), moves)
        want = fork_ref(self.np_pages, self.table, self.lens, self.refs, parents, children)
        self.same(moves, want)

    def same(self, moves, want):
        torch.cuda.synchronize()
        assert np.array_equal(moves.cpu().numpy(), want)
        for got, ref in zip(self.dev, (self.table, self.lens, self.refs)):
            assert np.array_equal(got.cpu().numpy(), ref)
        for got, ref in zip(self.pages, self.np_pages):
            assert np.array_equal(got.cpu().numpy(), ref)


def test_resize_gives_and_takes():
    tq = _tq()
    p = Pool(5, 8, 40, reserve=[0, 3, 7])
    for new in ([1, 16, 17, 0, 100], [2, 16, 18, 128, 99], [0, 0, 0, 128, 1], [128, 0, 5, 0, 1], [0] * 5):
        p.resize(tq, new)
    assert tq.get_device_error() == 0


def test_resize_refuses_what_does_not_fit_and_serves_the_rest():
    tq = _tq()
    p = Pool(4, 8, 10)
    p.resize(tq, [48, 16, 0, 0])
    assert tq.get_device_error() == 0
    p.resize(tq, [32, 128, 20, 0])          # 7 pages asked with 6 free: refused; the one after it too
    assert tq.get_device_error() == tq.DEVERR_NO_PAGES
    p.resize(tq, [32, 16, 100, 0])          # 7 free: fits exactly
    assert tq.get_device_error() == 0
    p.resize(tq, [32, 17, 0, 0])            # what a call releases is free for the next one
    assert tq.get_device_error() == tq.DEVERR_NO_PAGES
    p.resize(tq, [32, 17, 0, 0])
    assert tq.get_device_error() == 0


def test_bad_lengths_leave_the_sequence():
    tq = _tq()
    p = Pool(3, 4, 20)
    p.resize(tq, [20, 30, 40])
    p.resize(tq, [65, -1, 41])
    assert tq.get_device_error() == tq.DEVERR_SEQLEN_RANGE
    p.resize(tq, [2147483647, 64, -2147483648])
    assert tq.get_device_error() == tq.DEVERR_SEQLEN_RANGE


def test_window_pages_are_released_once():
    tq = _tq()
    p = Pool(3, 40, 150)
    p.resize(tq, [600, 100, 30])
    for new in ([601, 101, 31], [640, 300, 32], [640, 301, 20], [10, 200, 0]):
        p.resize(tq, new, window=100, sinks=20)
    p.resize(tq, [640, 400, 300], window=1, sinks=0)
    p.resize(tq, [0, 0, 0])
    assert np.all(p.refs == 0)
    assert tq.get_device_error() == 0


def test_fork_shares_and_copies():
    tq = _tq()
    p = Pool(8, 8, 60, layers=3)
    p.resize(tq, [40, 32, 0, 0, 0, 0, 0, 0])
    p.fork(tq, [0, 0, 1, 2], [2, 3, 4, 5])              # an empty parent, one whose last page is full
    assert tq.get_device_error() == 0
    p.fork(tq, [0, 7, 4], [7, 6, 5])                    # 7 is a child: empty at the start of the call
    assert tq.get_device_error() == 0
    # copy on write: cut a child into a shared page, then let it grow
    p.resize(tq, [40, 32, 10, 20, 30, 32, 0, 40])
    p.resize(tq, [41, 40, 11, 60, 33, 32, 3, 64])
    p.resize(tq, [0] * 8)
    assert np.all(p.refs == 0)
    assert tq.get_device_error() == 0


def test_fork_refusals():
    tq = _tq()
    p = Pool(6, 4, 8)
    p.resize(tq, [40, 20, 0, 0, 0, 0])                  # 5 pages, 3 free
    p.fork(tq, [0, 0, 9, -1, 1, 0, 0], [2, 2, 3, 4, 0, 6, -3])   # named twice, indices, a child in use
    assert tq.get_device_error() == tq.DEVERR_SEQ_INDEX
    p.fork(tq, [0, 1, 0], [3, 4, 5])                    # 2 free pages for three copies
    assert tq.get_device_error() == tq.DEVERR_NO_PAGES
    p.resize(tq, [0] * 6)
    assert np.all(p.refs == 0)


def test_entries_out_of_range_are_reported_and_skipped():
    tq = _tq()
    p = Pool(2, 4, 12)
    p.resize(tq, [40, 0])
    for x in (p.table, p.dev[0]):
        x[0, 0] = 12
        x[0, 2] = 5000                                  # the partly filled last page
    p.fork(tq, [0], [1])
    assert tq.get_device_error() == tq.DEVERR_BLOCK_RANGE
    p.resize(tq, [41, 0])
    assert tq.get_device_error() == tq.DEVERR_BLOCK_RANGE
    p.resize(tq, [0, 0])
    assert tq.get_device_error() == tq.DEVERR_BLOCK_RANGE


@pytest.mark.parametrize("batch,cols,pool,seed", [(4, 6, 30, 1), (50, 20, 500, 2), (300, 40, 9000, 3),
                                                  (33, 600, 70001, 4), (1500, 3, 4000, 5)])
def test_random_runs(batch, cols, pool, seed):
    """Random resizes and forks, pools of one CTA and of a whole cluster, odd sizes."""
    tq = _tq()
    rng = random.Random(seed)
    p = Pool(batch, cols, pool, layers=1, seed=seed, reserve=rng.sample(range(pool), pool // 7))
    for step in range(8):
        new = [rng.choice((int(n), rng.randrange(cols * BS + 1), min(cols * BS, int(n) + 1), 0)) for n in p.lens]
        p.resize(tq, new, window=rng.choice((0, 0, 50)), sinks=rng.choice((0, 17)))
        empty = [b for b in range(batch) if p.lens[b] == 0]
        children = rng.sample(empty, len(empty) // 2)
        if children:
            p.fork(tq, [rng.randrange(batch) for _ in children], children)
    assert tq.get_device_error() in (0, tq.DEVERR_NO_PAGES)


@pytest.mark.parametrize("layers", [1, 3])
@pytest.mark.parametrize("batch,length,keep", [(1, 1, 1), (3, 100, 33), (2, 700, 700), (5, 300, 0)])
def test_compact(layers, batch, length, keep):
    tq = _tq()
    rng = np.random.default_rng(length + keep)
    p = Pool(2 * batch, pages_of(length) + 2, 2 * batch * (pages_of(length) + 2), layers, seed=3)
    p.resize(tq, [length] * batch + [max(keep, 1)] * batch)
    counts = rng.integers(keep // 2, keep + 1, batch).astype(np.int32)
    counts[0] = keep
    pos = np.full((batch, keep + 3), -1, np.int32)
    for b in range(batch):
        some = rng.permutation(length)[:counts[b]]
        pos[b, :counts[b]] = np.sort(some) if b % 2 == 0 else some
    t, l, _ = p.dev
    tq.pages_compact(p.pages, t[:batch], l[:batch], p.i32(pos), p.i32(counts), t[batch:])
    compact_ref(p.np_pages, p.table[:batch], p.lens[:batch], pos, counts, p.table[batch:])
    p.same(p.i32([[0, 0]]), np.zeros((1, 2), np.int32))
    assert tq.get_device_error() == 0


def test_compact_skips_what_is_out_of_range():
    tq = _tq()
    p = Pool(6, 6, 60, layers=1, seed=3)
    p.resize(tq, [90, 90, 90, 40, 40, 40])
    for x in (p.table, p.dev[0]):
        x[1, 2] = -1
        x[2, 0] = 60
        x[5, 1] = 77
    pos = np.tile(np.arange(0, 80, 2, dtype=np.int32), (3, 1))
    pos[0, 5], pos[0, 6] = 90, -1
    t, l, _ = p.dev

    def run(counts, lens=None):
        ln = p.lens[:3] if lens is None else np.asarray(lens, np.int32)
        c = np.asarray(counts, np.int32)
        tq.pages_compact(p.pages, t[:3], p.i32(ln), p.i32(pos), p.i32(c), t[3:])
        compact_ref(p.np_pages, p.table[:3], ln, pos, c, p.table[3:])
        p.same(p.i32([[0, 0]]), np.zeros((1, 2), np.int32))
        return tq.get_device_error()

    assert run([40, 40, 40]) == tq.DEVERR_SLOT_RANGE | tq.DEVERR_BLOCK_RANGE
    assert run([41, -1, 0]) == tq.DEVERR_SEQLEN_RANGE
    assert run([3, 3, 0], [97, -1, 5]) == tq.DEVERR_SEQLEN_RANGE


def test_page_operations_captured():
    """A graph of one decode step's page work, replayed: state advances as the calls would."""
    tq = _tq()
    p = Pool(6, 10, 80, layers=2)
    p.resize(tq, [20, 31, 47, 0, 0, 0])
    t, l, r = p.dev
    moves, fmoves = p.i32(np.zeros((6, 2))), p.i32(np.zeros((2, 2)))
    new, parents, children = p.i32([0] * 6), p.i32([0, 1]), p.i32([3, 4])
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        tq.pages_resize(p.pages, t, l, new, r, moves)
        tq.pages_fork(p.pages, t, l, r, parents, children, fmoves)
    for step in range(4):
        goal = [21 + step, 33 + step, 48, 0, 0, 0]
        new.copy_(p.i32(goal))
        g.replay()
        want = resize_ref(p.np_pages, p.table, p.lens, goal, p.refs)
        fork_want = fork_ref(p.np_pages, p.table, p.lens, p.refs, [0, 1], [3, 4])
        p.same(moves, want)
        assert np.array_equal(fmoves.cpu().numpy(), fork_want)
    assert tq.get_device_error() == 0


def test_a_serving_run():
    """Admit prompts, append and attend by chunks, fork one, decode both with a window (each its own
    token), release pages out of the window, cut one sequence to its kept tokens: every output against
    the definition over the pages as they are."""
    tq = _tq()
    d, hq, hkv, kb, vb, seed = 128, 8, 2, 4, 4, 11
    scale = d ** -0.5
    cb = tq.load_codebooks(d, kb, vb, "cuda")
    g = torch.Generator().manual_seed(1)
    pool, cols, batch = 64, 20, 4
    pages = torch.zeros(pool, BS, hkv, tq.slot_bytes(d, kb, vb), dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")     # noqa: E731
    table = torch.full((batch, cols), -1, dtype=torch.int32, device="cuda")
    lens, refs, moves = i32([0] * batch), i32([0] * pool), i32([[0, 0]] * batch)

    def append(old):
        """The new tokens of each sequence, random K and V, to their slots."""
        slots = []
        for b, n in enumerate(lens.tolist()):
            row = table[b].tolist()
            slots += [row[t // BS] * BS + t % BS for t in range(old[b], n)]
        k, v = (torch.randn(len(slots), hkv, d, generator=g).bfloat16().cuda() for _ in range(2))
        tq.quantize_append(pages, torch.tensor(slots, device="cuda"), k, v, cb, seed)

    def attend(q_lens, window=0, sinks=0, single=False):
        starts = np.concatenate([[0], np.cumsum(q_lens)])
        q = torch.randn(int(starts[-1]), hq, d, generator=g).bfloat16().cuda()
        out = torch.empty_like(q)
        if single:
            tq.paged_decode_window(out, q, pages, table, lens, cb, seed, scale, window, sinks)
        else:
            tq.paged_attend(out, q, i32(starts.tolist()), pages, table, lens, cb, seed, scale, int(max(q_lens)),
                            window, sinks)
        ref, tol = attend_ref(to_np_f64(q), starts, pages.cpu().numpy(), table.cpu().numpy(), lens.cpu().numpy(), d,
                              kb, vb, seed, scale, window, sinks, out_eps(torch.bfloat16))
        check_rows(to_np_f64(out), ref, tol)

    for new, q_lens in (([60, 33, 0, 0], [60, 33, 0, 0]), ([200, 34, 0, 0], [140, 1, 0, 0])):
        old = lens.tolist()
        tq.pages_resize(pages, table, lens, i32(new), refs, moves)
        append(old)
        attend(q_lens)
    tq.pages_fork(pages, table, lens, refs, i32([0, 1]), i32([2, 3]), i32([[0, 0]] * 2))
    assert lens.tolist() == [200, 34, 200, 34]
    for _ in range(20):
        old = lens.tolist()
        tq.pages_resize(pages, table, lens, lens + 1, refs, moves, window=48, sinks=4)
        append(old)
        attend([1] * 4, 48, 4, single=True)
    row = table[0].tolist()
    assert row[0] >= 0 and row[2] == -1 and refs.sum().item() == (table >= 0).sum().item()
    # sequence 1 keeps its first 4 and every third token, in the pages of a new row
    n = int(lens[1])
    keep = [t for t in range(n) if t < 4 or t % 3 == 0]
    dst, dlens = torch.full((1, cols), -1, dtype=torch.int32, device="cuda"), i32([0])
    tq.pages_resize(pages, dst, dlens, i32([len(keep)]), refs, moves[:1])
    tq.pages_compact(pages, table[1:2], lens[1:2], i32([keep]), i32([len(keep)]), dst)
    tq.pages_resize(pages, table, lens, i32([0 if b == 1 else int(x) for b, x in enumerate(lens)]), refs, moves)
    table[1], lens[1] = dst[0], dlens[0]
    assert tq.get_device_error() == 0
    # without a window the rows of sequences 0 and 2 reach released pages: skipped, and reported
    attend([2, 5, 1, 3])
    assert tq.get_device_error() == tq.DEVERR_BLOCK_RANGE
    tq.pages_resize(pages, table, lens, i32([0] * batch), refs, moves)
    assert torch.all(refs == 0) and torch.all(table == -1)
    assert tq.get_device_error() == 0
