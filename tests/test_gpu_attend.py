"""GPU parity of tq_paged_attend and tq_paged_decode_window with the definition in 64 bits, over
pages that tq_quantize_append wrote, at the lengths, masks, layouts and values where they can go
wrong."""
import numpy as np
import pytest
import torch

from oracle import tq_oracle as O
from kv_cache_vector_append_b200 import workloads as W
from tests.attend_helpers import BS, attend_ref, check_rows, out_eps
from tests.gpu_helpers import gpu_append, gpu_decode, require_gpu, to_np_f64

pytestmark = pytest.mark.gpu
SEED = 77
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _tq():
    require_gpu()
    import kv_cache_vector_append_b200 as tq
    return tq


class Case:
    """Packed pages of sequences of the given lengths and queries for their last tokens."""

    def __init__(self, tq, d, hq, hkv, kb, vb, lens, q_lens, dtype="bf16", seed=5, slot_stride=None):
        spec = W.WorkloadSpec("attend", d, hq, hkv, len(lens), kb, vb, "bfloat16", seq_len=max(max(lens), 1),
                              n_outliers=2, outlier_factor=10.0, seed=seed, sign_seed=SEED)
        wl = W.generate(spec)
        self.tq, self.spec, self.scale = tq, spec, spec.scale
        self.pages, self.cb = gpu_append(tq, wl, slot_stride=slot_stride)
        self.table = torch.from_numpy(wl.block_table).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        starts = np.concatenate([[0], np.cumsum(q_lens)])
        self.max_q = int(max(q_lens))
        self.starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        g = torch.Generator().manual_seed(seed)
        self.q = torch.randn(int(starts[-1]), hq, d, generator=g).to(DT[dtype]).cuda()
        self.out = torch.full_like(self.q, 7.0)

    def run(self, window=0, sinks=0, stream=None):
        self.tq.paged_attend(self.out, self.q, self.starts, self.pages, self.table, self.lens, self.cb, SEED,
                             self.scale, self.max_q, window=window, sinks=sinks, stream=stream)
        return self.out

    def ref(self, window=0, sinks=0, starts=None):
        s = self.spec
        return attend_ref(to_np_f64(self.q), self.starts.cpu().numpy() if starts is None else starts,
                          self.pages.cpu().numpy(), self.table.cpu().numpy(), self.lens.cpu().numpy(), s.head_dim,
                          s.k_bits, s.v_bits, SEED, self.scale, window, sinks, out_eps(self.out.dtype))

    def check(self, window=0, sinks=0, together=False):
        got = to_np_f64(self.run(window, sinks))
        torch.cuda.synchronize()
        return check_rows(got, *self.ref(window, sinks), out_eps(self.out.dtype) if together else None)


# lengths around the page and tile borders, new tokens from none to all of the sequence
GEOMETRIES = [
    # d, hq, hkv, kb, vb, lens, q_lens, window, sinks, dtype
    (128, 8, 2, 4, 4, [1, 16, 17, 300], [1, 1, 1, 1], 0, 0, "bf16"),
    (128, 8, 2, 4, 4, [1, 15, 129, 0, 64], [1, 3, 129, 0, 64], 0, 0, "bf16"),
    (128, 28, 4, 4, 2, [200, 5, 131], [70, 5, 2], 0, 0, "f16"),
    (128, 4, 4, 3, 2, [257, 128], [257, 127], 0, 0, "bf16"),
    (64, 14, 2, 8, 8, [90, 400, 33], [4, 4, 3], 0, 0, "bf16"),
    (64, 2, 2, 2, 3, [513], [300], 0, 0, "f16"),
    (256, 4, 2, 4, 4, [150, 64, 65], [40, 64, 1], 0, 0, "bf16"),
    (256, 2, 1, 8, 8, [140], [70], 0, 0, "f32"),
    (128, 16, 1, 4, 4, [100, 3], [9, 3], 0, 0, "f16"),
    (128, 40, 2, 4, 4, [60, 33], [2, 33], 0, 0, "bf16"),
    # windows: of one token, inside a page, at a page's border, over tiles; sinks inside the window too
    (128, 8, 2, 4, 4, [300, 40, 17], [20, 40, 1], 1, 0, "bf16"),
    (128, 8, 2, 4, 4, [300, 40, 1], [130, 3, 1], 16, 1, "bf16"),
    (128, 8, 2, 4, 2, [1000, 400, 35], [300, 1, 2], 100, 4, "f16"),
    (64, 14, 2, 8, 8, [700, 100], [33, 100], 128, 20, "bf16"),
    (256, 4, 2, 3, 4, [420], [150], 33, 17, "bf16"),
    (128, 4, 1, 4, 4, [900], [260], 150, 200, "bf16"),
    # keys split over several blocks: one and two row tiles, few rows, odd ends
    (128, 8, 2, 4, 4, [5001, 2100], [20, 41], 0, 0, "bf16"),
    (128, 8, 2, 3, 2, [4100], [200], 0, 0, "f16"),
    (128, 8, 2, 8, 8, [3333], [130], 2000, 5, "bf16"),
    (64, 14, 2, 8, 8, [3500, 77], [11, 60], 0, 0, "bf16"),
    (256, 4, 2, 4, 3, [2600], [50], 0, 0, "bf16"),
    (128, 8, 2, 4, 2, [3000, 4000], [8, 3], 0, 0, "f32"),
    (256, 4, 2, 8, 2, [2000], [3], 0, 0, "f16"),
]


@pytest.mark.parametrize("d,hq,hkv,kb,vb,lens,q_lens,window,sinks,dtype", GEOMETRIES)
def test_attend_against_the_definition(d, hq, hkv, kb, vb, lens, q_lens, window, sinks, dtype):
    tq = _tq()
    Case(tq, d, hq, hkv, kb, vb, lens, q_lens, dtype).check(window, sinks, together=True)
    assert tq.get_device_error() == 0


@pytest.mark.parametrize("kb", [2, 3, 4, 8])
@pytest.mark.parametrize("vb", [2, 3, 4, 8])
@pytest.mark.parametrize("d,q_lens", [(64, [2, 30]), (128, [1, 41]), (256, [2, 20])])
def test_every_width_pair(kb, vb, d, q_lens):
    tq = _tq()
    Case(tq, d, 4, 2, kb, vb, [150, 61], q_lens, "bf16", seed=kb * 10 + vb).check()
    Case(tq, d, 4, 2, kb, vb, [150, 61], q_lens, "bf16", seed=kb * 10 + vb).check(37, 3)


@pytest.mark.parametrize("d,hq,hkv,kb,vb", [(128, 32, 8, 4, 4), (128, 28, 4, 4, 2), (64, 14, 2, 8, 8),
                                            (256, 16, 4, 4, 4), (128, 16, 1, 3, 2)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 4), (1000, 1), (1 << 30, 0)])
def test_decode_window_against_the_definition(d, hq, hkv, kb, vb, window, sinks):
    tq = _tq()
    lens = [1, 63, 64, 65, 0, 1100, 333]
    c = Case(tq, d, hq, hkv, kb, vb, lens, [1] * len(lens))
    tq.paged_decode_window(c.out, c.q, c.pages, c.table, c.lens, c.cb, SEED, c.scale, window, sinks)
    check_rows(to_np_f64(c.out), *c.ref(window, sinks), out_eps(c.out.dtype))
    # the same as a chunk of one token each
    one = c.out.clone()
    assert torch.equal(one, c.run(window, sinks))
    assert tq.get_device_error() == 0


def test_one_token_without_a_window_is_the_whole_sequence_decode():
    tq = _tq()
    lens = [300, 17, 64, 1, 2000, 0]
    spec = W.WorkloadSpec("d", 128, 8, 2, len(lens), 4, 4, "bfloat16", seq_len=2000, seed=3, sign_seed=SEED)
    wl = W.generate(spec)
    wl.seq_lens = np.asarray(lens, np.int32)
    pages, cb = gpu_append(tq, wl)
    want = to_np_f64(gpu_decode(tq, wl, pages, cb, torch.float32))
    c = Case(tq, 128, 8, 2, 4, 4, lens, [1] * len(lens))
    c.pages, c.cb, c.table, c.q = pages, cb, torch.from_numpy(wl.block_table).cuda(), wl.q.cuda()
    c.out = torch.empty(c.q.shape, dtype=torch.float32, device="cuda")
    _, tol = c.ref()
    check_rows(to_np_f64(c.run()), want, 2 * tol)       # both are within tol of the definition


def test_rows_before_the_first_token_and_rows_of_no_sequence():
    tq = _tq()
    c = Case(tq, 128, 8, 2, 4, 4, [5, 40, 0, 200], [9, 3, 2, 66])      # 4 rows before token 0; 2 of an empty one
    starts = c.starts.cpu().numpy()
    wide = torch.full((c.q.shape[0] + 7, 8, 128), 7.0, dtype=c.q.dtype, device="cuda")
    q = wide.clone()
    q[3:-4] = c.q
    c.q, c.out = q, wide
    c.starts = c.starts + 3
    got = to_np_f64(c.run())
    ref, tol = c.ref()
    assert np.all(got[:3] == 7.0) and np.all(got[-4:] == 7.0)
    sl = slice(3, -4)
    check_rows(got[sl], ref[sl], tol[sl])
    assert np.all(got[3:3 + 4] == 0.0) and np.all(got[3 + starts[2]:3 + starts[3]] == 0.0)
    assert tq.get_device_error() == 0


@pytest.mark.parametrize("q_lens", [[1, 1], [2, 1], [40, 90]])
def test_strided_tensors_and_interleaved_layers(q_lens):
    tq = _tq()
    c = Case(tq, 128, 4, 2, 4, 2, [100, 90], q_lens, slot_stride=112)
    want = to_np_f64(c.run(0, 0)).copy()
    ref, tol = c.ref()
    check_rows(want, ref, tol)
    # q and out: slices of wider tensors; the pool: one of three layers of each block, heads before
    # tokens in a page, blocks of the table in a wider row
    q = torch.randn(c.q.shape[0], 3, 4, 160, device="cuda").to(c.q.dtype)
    q[:, 1, :, 8:136] = c.q
    out = torch.full((c.q.shape[0], 4, 2, 136), 7.0, dtype=c.q.dtype, device="cuda")
    pool = torch.full((c.pages.shape[0], 3, 2, BS, 112), 255, dtype=torch.uint8, device="cuda")
    pool[:, 1] = c.pages.permute(0, 2, 1, 3)
    table = torch.full((2, c.table.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    tq.paged_attend(out[:, :, 1, 4:132], q[:, 1, :, 8:136], c.starts, pool[:, 1].permute(0, 2, 1, 3),
                    table[:, :c.table.shape[1]], c.lens, c.cb, SEED, c.scale, c.max_q)
    assert np.array_equal(to_np_f64(out[:, :, 1, 4:132]), want)
    assert torch.all(out[:, :, 0] == 7.0) and torch.all(out[:, :, 1, :4] == 7.0)


@pytest.mark.parametrize("q_lens,window,sinks", [([1, 1], 40, 4), ([1, 2], 40, 20), ([50, 70], 40, 4),
                                                 ([50, 70], 0, 0)])
def test_unseen_tokens_may_hold_anything(q_lens, window, sinks):
    """Tokens behind the sequence's end, and those no row sees, have NaN norms, entries of released
    pages are -1; in a chunk the later tokens' NaN values reach the rows that see them only."""
    tq = _tq()
    lens = [300, 277]
    c = Case(tq, 128, 8, 2, 4, 4, lens, q_lens)
    pages = c.pages.cpu().numpy()
    kreg = O.region_bytes(128, 4)
    nan = np.frombuffer(np.float32(np.nan).tobytes(), np.uint8)
    table = c.table.cpu().numpy()
    full = 304
    for b, n in enumerate(lens):
        p0 = n - q_lens[b]
        for t in range(full):
            unseen = t >= n or (window and sinks <= t <= p0 - window)
            late = t == n - 1 and q_lens[b] > 1                     # the last token poisons its own row only
            if unseen or late:
                page = table[b, t // BS]
                pages[page, t % BS, :, kreg - 4:kreg] = nan
                pages[page, t % BS, :, 2 * kreg - 4:2 * kreg] = nan
        if window:
            for col in range((full + BS - 1) // BS):
                if col * BS >= sinks and (col + 1) * BS <= p0 - window + 1:
                    table[b, col] = -1
    c.pages = torch.from_numpy(pages).cuda()
    c.table = torch.from_numpy(table).cuda()
    c.check(window, sinks)
    assert tq.get_device_error() == 0


@pytest.mark.parametrize("n,longest,q_len", [(170, 5000, 1), (40, 5000, 70), (20, 2500, 70), (40, 700, 6)])
def test_many_sequences(n, longest, q_len):
    """More and fewer sequences than a warp ranks, one of them far longer than the others."""
    tq = _tq()
    rng = np.random.default_rng(n)
    lens = rng.integers(1, 90, n)
    lens[n // 3] = longest
    q_lens = np.minimum(rng.integers(0, 4, n), lens)
    q_lens[n // 3], q_lens[0] = q_len, min(q_len, lens[0])
    c = Case(tq, 128, 8, 2, 4, 2, lens.tolist(), q_lens.tolist())
    c.check()
    c.check(300, 3)
    assert tq.get_device_error() == 0


@pytest.mark.parametrize("q_lens", [[1, 2], [7, 3], [90, 40]])
@pytest.mark.parametrize("scale", [-0.07, 0.0, 1e-30])
def test_scales_of_either_sign(q_lens, scale):
    tq = _tq()
    c = Case(tq, 128, 8, 2, 4, 4, [300, 100], q_lens)
    c.scale = scale
    c.check()
    c.check(50, 3)


@pytest.mark.parametrize("q_lens", [[1, 2], [7, 3], [90, 40]])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rows_at_odd_addresses(q_lens, dtype):
    """q and out whose rows start on no 16-byte boundary, both as q's type and as f32."""
    tq = _tq()
    c = Case(tq, 128, 8, 2, 4, 4, [300, 100], q_lens, dtype)
    want = c.run().clone()
    n = c.q.shape[0]
    q = torch.zeros(n, 8, 133, dtype=c.q.dtype, device="cuda")[:, :, 3:131]
    q.copy_(c.q)
    for out_dtype in (c.q.dtype, torch.float32):
        out = torch.zeros(n, 8, 131, dtype=out_dtype, device="cuda")[:, :, 1:129]
        tq.paged_attend(out, q, c.starts, c.pages, c.table, c.lens, c.cb, SEED, c.scale, c.max_q)
        assert torch.equal(out.to(c.q.dtype), want)


@pytest.mark.parametrize("q_lens", [[1, 2], [90, 40]])
def test_broadcast_queries(q_lens):
    """One query row for all heads (a dim of stride 0), and out head by head apart."""
    tq = _tq()
    c = Case(tq, 128, 8, 2, 4, 4, [300, 100], q_lens)
    n = c.q.shape[0]
    c.q = c.q[:, :1].expand(n, 8, 128)
    want = c.run().clone()
    check_rows(to_np_f64(want), *c.ref())
    out = torch.zeros(8, n, 128, dtype=c.q.dtype, device="cuda").transpose(0, 1)
    tq.paged_attend(out, c.q, c.starts, c.pages, c.table, c.lens, c.cb, SEED, c.scale, c.max_q)
    assert torch.equal(out, want)


@pytest.mark.parametrize("rows", [1, 3, 40])
def test_a_bad_entry_skips_its_page(rows):
    tq = _tq()
    c = Case(tq, 128, 4, 2, 4, 4, [200, 90], [rows, rows])
    c.table[0, 3] = c.pages.shape[0]
    c.table[1, 0] = -5
    c.check()
    assert tq.get_device_error() == tq.DEVERR_BLOCK_RANGE
    c.table[0, 3] = 1
    c.table[1, 0] = 2
    c.check()
    assert tq.get_device_error() == 0


@pytest.mark.parametrize("rows", [1, 40])
def test_bad_lengths_and_ranges(rows):
    tq = _tq()
    c = Case(tq, 128, 4, 2, 4, 4, [60, 60, 60], [rows] * 3)
    good = c.run().clone()
    c.lens[1] = 60 * 1000
    c.out.fill_(7.0)
    c.run()
    assert tq.get_device_error() == tq.DEVERR_SEQLEN_RANGE
    assert torch.equal(c.out[:rows], good[:rows]) and torch.equal(c.out[2 * rows:], good[2 * rows:])
    assert torch.all(c.out[rows:2 * rows] == 0)
    c.lens[1] = 60
    for bad in ([0, rows, 3 * rows + 1, 3 * rows], [0, rows, -1, 3 * rows], [-4, rows, 2 * rows, 3 * rows]):
        c.starts.copy_(torch.tensor(bad, dtype=torch.int32))
        c.out.fill_(7.0)
        c.run()
        assert tq.get_device_error() == tq.DEVERR_SEQLEN_RANGE
        for b in range(3):
            mine = c.out[b * rows:(b + 1) * rows]
            if bad[b:b + 2] == [b * rows, (b + 1) * rows]:
                assert torch.equal(mine, good[b * rows:(b + 1) * rows])
            elif not (0 <= bad[b] <= bad[b + 1] <= 3 * rows):
                assert torch.all(mine == 7.0)
    # more new tokens than max_q says: that sequence is left out
    c.starts.copy_(torch.tensor([0, rows, 3 * rows, 3 * rows], dtype=torch.int32))
    c.out.fill_(7.0)
    c.run()
    assert tq.get_device_error() == tq.DEVERR_SEQLEN_RANGE
    assert torch.equal(c.out[:rows], good[:rows]) and torch.all(c.out[rows:] == 7.0)


@pytest.mark.parametrize("q_len", [1, 50])
@pytest.mark.parametrize("kf,vf", [(1.0, 1e-20), (1e-30, 1e25), (3e5, 1.0), (0.0, 0.0)])
def test_norms_far_from_one(q_len, kf, vf):
    """Norms scaled by large and small factors (all, and of every third token alone)."""
    tq = _tq()
    for every in (1, 3):
        c = Case(tq, 128, 4, 2, 4, 4, [140], [q_len], "f32")
        kreg = O.region_bytes(128, 4)
        pages = c.pages.cpu().numpy()
        for off, f in ((kreg - 4, kf), (2 * kreg - 4, vf)):
            norm = np.ascontiguousarray(pages[..., off:off + 4]).view(np.float32)
            norm[:, ::every] = norm[:, ::every] * np.float32(f)
            pages[..., off:off + 4] = norm.view(np.uint8)
        c.pages = torch.from_numpy(pages).cuda()
        if kf > 1:
            c.scale = 1.0 / (kf * 128 ** 0.5)
        got = to_np_f64(c.run())
        ref, tol = c.ref()
        big = max(1.0, float(np.abs(ref).max()))
        check_rows(got / big, ref / big, tol / big)


def test_zero_queries_and_flat_scores():
    tq = _tq()
    c = Case(tq, 128, 4, 2, 4, 4, [77, 200], [3, 60])
    c.q.zero_()
    c.check()
    c.check(10, 2)


def test_blocks_past_four_gigabytes():
    """Pages at byte offsets over 2^32, rows and heads as usual."""
    tq = _tq()
    for q_lens in ([1, 1], [50, 3]):
        c = Case(tq, 128, 8, 2, 4, 4, [100, 64], q_lens)
        want = c.run().clone()
        n = (1 << 32) // (BS * 2 * 136) + 40
        pool = torch.zeros(n, BS, 2, 136, dtype=torch.uint8, device="cuda")
        k = c.pages.shape[0]
        pool[n - k:] = c.pages
        c.pages = pool
        c.table = torch.where(c.table >= 0, c.table + (n - k), c.table)
        assert torch.equal(c.run(), want)


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [5, 2, 70]])
def test_captured_replayed_and_on_other_streams(q_lens):
    tq = _tq()
    lens = [300, 77, 90]
    a = Case(tq, 128, 8, 2, 4, 4, lens, q_lens)
    b = Case(tq, 128, 8, 2, 4, 4, lens, q_lens, seed=9)
    a_want, b_want = a.run(64, 4).clone(), b.run().clone()
    graphs = []
    for c, args in ((a, (64, 4)), (b, (0, 0))):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                c.run(*args)
        graphs.append(g)
    torch.cuda.synchronize()
    a.out.fill_(7.0)
    b.out.fill_(7.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):                                       # both graphs at once: nothing is shared
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.out, a_want) and torch.equal(b.out, b_want)
    # a replay reads the tables and lengths of its own time
    a.lens.copy_(torch.tensor([290, 76, 80], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    check_rows(to_np_f64(a.out), *a.ref(64, 4))


def test_same_bits_every_time():
    tq = _tq()
    c = Case(tq, 128, 28, 4, 4, 2, [3000, 500], [1, 130])
    first = c.run().clone()
    for _ in range(5):
        assert torch.equal(c.run(), first)
