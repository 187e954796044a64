"""Which tokens a row sees, one by one: keys of norm 0 give every visible token the same weight, values
of one direction whose norms stand out every few tokens show a token, a page or a split too many or
too few in the rows at whose edge it lies."""
import numpy as np
import pytest
import torch

from oracle import tq_oracle as O
from tests.attend_helpers import BS
from tests.gpu_helpers import oracle_table, to_np_f64
from tests.test_gpu_attend import SEED, Case, _tq

pytestmark = pytest.mark.gpu


class Edges:
    """Sequences of equal keys; token t's value is norm[t] times the direction of its head."""

    def __init__(self, tq, d, hq, hkv, kb, vb, lens, q_lens, heavy, every, extra_cols=0):
        rng = np.random.default_rng(d + kb * 10 + vb)
        self.tq, self.d, self.hq, self.hkv, self.lens = tq, d, hq, hkv, lens
        kreg, vreg = O.region_bytes(d, kb), O.region_bytes(d, vb)
        cols = max((max(lens) + BS - 1) // BS, 1) + extra_cols
        nblk = [(n + BS - 1) // BS for n in lens]
        order = rng.permutation(sum(nblk) + 3)
        self.table = np.full((len(lens), cols), -1, np.int32)
        self.norm = np.where(np.arange(cols * BS) % every == 0, float(heavy), 1.0)
        stride = (kreg + vreg + 7) // 8 * 8
        pages = rng.integers(0, 256, (len(order), BS, hkv, stride), dtype=np.uint8)
        code = rng.integers(0, 256, (hkv, vreg - 4), dtype=np.uint8)
        pages[..., kreg - 4:kreg] = 0                       # key norms
        pages[..., kreg:kreg + vreg - 4] = code
        at = 0
        for b, n in enumerate(nblk):
            self.table[b, :n] = order[at:at + n]
            at += n
            for c in range(n):
                norm = self.norm[c * BS:(c + 1) * BS].astype(np.float32)
                pages[self.table[b, c], :, :, kreg + vreg - 4:kreg + vreg] = norm.view(np.uint8).reshape(BS, 1, 4)
        vi, _ = O.decode_region(pages[0, 0, :, kreg:kreg + vreg], d, vb)
        self.value = O.dequantize_rows(vi, np.ones(hkv), oracle_table(d, vb), O.rht_signs(d, SEED))   # [H_kv, D]
        self.pages = torch.from_numpy(pages).cuda()
        self.starts = np.concatenate([[0], np.cumsum(q_lens)])
        self.max_q = int(max(q_lens))
        g = torch.Generator().manual_seed(1)
        self.q = torch.randn(int(self.starts[-1]), hq, d, generator=g).cuda()
        self.cb = tq.load_codebooks(d, kb, vb, "cuda")

    def check(self, window, sinks, single=False):
        i32 = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()       # noqa: E731
        out = torch.full_like(self.q, 7.0)
        table, lens = i32(self.table), i32(self.lens)
        if single:
            self.tq.paged_decode_window(out, self.q, self.pages, table, lens, self.cb, SEED, 1.0, window, sinks)
        else:
            self.tq.paged_attend(out, self.q, i32(self.starts), self.pages, table, lens, self.cb, SEED, 1.0,
                                 self.max_q, window=window, sinks=sinks)
        mean = np.zeros(out.shape[0])
        for b, n in enumerate(self.lens):
            there = np.repeat((self.table[b] >= 0) & (self.table[b] < self.pages.shape[0]), BS)
            t = np.arange(len(there))
            for i in range(self.starts[b], self.starts[b + 1]):
                p = n - int(self.starts[b + 1]) + i
                see = there & (t <= p) & ((t > p - window) | (t < sinks) if window else True)
                mean[i] = self.norm[see].mean() if see.any() else 0.0
        head = np.arange(self.hq) // (self.hq // self.hkv)
        ref = mean[:, None, None] * self.value[head]
        err = np.linalg.norm(to_np_f64(out) - ref, axis=-1)
        # centroids, norms (or weights times norms) and their product are rounded to fp16, 2^-11 each;
        # all values have one direction, so nothing cancels.  1e-5: sums in fp32
        allowed = (3 * 2.0 ** -11 + 1e-5) * np.linalg.norm(ref, axis=-1)
        assert np.all(err <= allowed), (window, sinks, np.argwhere(err > allowed)[:6].tolist())


MASKS = [(0, 0), (1, 0), (1, 1), (2, 5), (15, 0), (16, 16), (17, 15), (33, 17), (100, 4), (128, 0), (300, 40)]


@pytest.mark.parametrize("heavy", [100, 1000])
@pytest.mark.parametrize("d,hq,hkv,kb,vb,lens,q_lens", [
    (128, 4, 2, 4, 4, [400, 37, 150], [16, 11, 15]),        # few rows: one to four row tiles
    (128, 4, 2, 4, 2, [333, 16, 17], [3, 1, 2]),
    (64, 14, 2, 8, 8, [290, 40], [4, 3]),
    (256, 4, 2, 3, 3, [260, 33], [9, 16]),
    (128, 8, 2, 4, 4, [500, 129, 64, 1], [70, 129, 9, 1]),  # tiles: one row tile and two a block
    (128, 16, 2, 3, 2, [450, 60], [75, 60]),
    (128, 4, 2, 8, 4, [450, 60], [40, 60]),                 # 64-key tiles
    (128, 8, 2, 8, 8, [450, 60], [90, 60]),
    (64, 8, 2, 2, 3, [400, 70], [80, 70]),
    (64, 14, 2, 8, 8, [400, 70], [80, 7]),
    (256, 4, 2, 4, 8, [330, 70], [80, 70]),
    (256, 4, 2, 8, 2, [330, 70], [80, 70]),                 # 32-key tiles
])
def test_what_a_row_sees(d, hq, hkv, kb, vb, lens, q_lens, heavy):
    tq = _tq()
    e = Edges(tq, d, hq, hkv, kb, vb, lens, q_lens, heavy, 7)
    for window, sinks in MASKS:
        e.check(window, sinks)
    assert tq.get_device_error() == 0


@pytest.mark.parametrize("d,kb,vb", [(64, 8, 8), (128, 4, 2), (128, 8, 3), (256, 4, 4), (256, 8, 8)])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [8, 2, 5], [100, 60, 5], [33, 1, 90]])
def test_every_page_of_a_long_sequence(d, kb, vb, q_lens):
    """Sequences split over blocks, in tables as wide as they need and wider."""
    tq = _tq()
    for extra in (0, 200):
        e = Edges(tq, d, 4, 2, kb, vb, [2500, 1000, 90], q_lens, 1000, 16, extra)
        for window, sinks in ((0, 0), (700, 33), (1030, 1)):
            e.check(window, sinks)
        e.table[0, [3, 50, 155]] = [-1, e.pages.shape[0], -7]
        e.check(0, 0)
        assert tq.get_device_error() == tq.DEVERR_BLOCK_RANGE


@pytest.mark.parametrize("d,kb,vb", [(64, 8, 8), (128, 4, 2), (256, 4, 4)])
def test_what_single_tokens_see(d, kb, vb):
    tq = _tq()
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 100, 255, 256, 257, 301, 0, 700]
    e = Edges(tq, d, 8, 2, kb, vb, lens, [1] * len(lens), 1000, 5)
    for window, sinks in MASKS[1:] + [(2**31 - 1, 2**31 - 1), (5, 2**31 - 1), (2**31 - 1, 0)]:
        e.check(window, sinks, single=True)
        e.check(window, sinks)
    assert tq.get_device_error() == 0


@pytest.mark.parametrize("n,longest,q_len", [(33, 3000, 1), (40, 2000, 60), (300, 500, 3)])
def test_many_sequences_see_their_own(n, longest, q_len):
    tq = _tq()
    rng = np.random.default_rng(n)
    lens = rng.integers(1, 90, n)
    lens[n // 2] = longest
    q_lens = np.minimum(rng.integers(0, 4, n), lens)
    q_lens[n // 2] = q_len
    e = Edges(tq, 128, 8, 2, 4, 2, lens.tolist(), q_lens.tolist(), 1000, 16)
    for window, sinks in ((0, 0), (50, 3)):
        e.check(window, sinks)
    assert tq.get_device_error() == 0


@pytest.mark.parametrize("q_lens", [[1, 2], [7, 3], [90, 40]])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_queries_that_are_no_numbers_stay_in_their_rows(q_lens, dtype):
    tq = _tq()
    c = Case(tq, 128, 8, 2, 4, 4, [300, 100], q_lens, dtype)
    want = c.run(60, 4).clone()
    rows = c.q.shape[0]
    bad = [(0, 0), (rows - 1, 7), (rows // 2, 3)]
    for (r, h), x in zip(bad, (float("nan"), float("inf"), -float("inf"))):
        c.q[r, h, 5] = x
    got = c.run(60, 4).clone()
    for r, h in bad:
        assert torch.all(torch.isnan(got[r, h]))
        got[r, h] = want[r, h]
    assert torch.equal(got, want)
    assert tq.get_device_error() == 0


@pytest.mark.parametrize("q_lens", [[1, 2], [90, 40]])
def test_unseen_tokens_of_infinite_norm(q_lens):
    """Norms of either infinity in every token that no row sees."""
    tq = _tq()
    lens, window, sinks = [300, 277], 40, 4
    c = Case(tq, 128, 8, 2, 4, 4, lens, q_lens, "f32")
    pages, table = c.pages.cpu().numpy(), c.table.cpu().numpy()
    kreg = O.region_bytes(128, 4)
    for b, n in enumerate(lens):
        for t in range(304):
            if t >= n or sinks <= t <= n - q_lens[b] - window:
                for off in (kreg, 2 * kreg):
                    inf = np.float32((-1) ** (t // 3) * np.inf)
                    pages[table[b, t // BS], t % BS, :, off - 4:off] = np.frombuffer(inf.tobytes(), np.uint8)
    c.pages = torch.from_numpy(pages).cuda()
    c.check(window, sinks)
    assert tq.get_device_error() == 0
