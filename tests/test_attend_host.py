"""What the new entry points refuse on the host, before anything is enqueued (no GPU needed)."""
import ctypes

import pytest
import torch

from tests.test_abi import _fake


def _lib():
    from kv_cache_vector_append_b200 import _binding as B
    return B, B._load()


def _books(B, d=128, kb=4, vb=4):
    c = B.CodebooksDesc()
    c.k = B.CodebookDesc(d, kb, 0x20000, 0x30000)
    c.v = B.CodebookDesc(d, vb, 0x40000, 0x50000)
    return c


def _attend(**kw):
    B, lib = _lib()
    a = dict(out=_fake([10, 8, 128], B.BF16), q=_fake([10, 8, 128], B.BF16), starts=_fake([3], B.I32),
             pages=_fake([4, 16, 2, 136], B.U8), table=_fake([2, 4], B.I32), lens=_fake([2], B.I32),
             cb=_books(B), scale=0.1, max_q=5, window=0, sinks=0)
    a.update(kw)
    return lib.tq_paged_attend(a["out"], a["q"], a["starts"], a["pages"], a["table"], a["lens"],
                               ctypes.byref(a["cb"]) if a["cb"] is not None else None, 0, a["scale"], a["max_q"],
                               a["window"], a["sinks"], None)


def test_attend_refusals():
    B, _ = _lib()
    bad, no = B.ERR_INVALID_ARG, B.ERR_UNSUPPORTED
    assert _attend(cb=None) == bad
    assert _attend(scale=float("inf")) == bad
    assert _attend(max_q=-1) == bad
    assert _attend(window=-1) == bad
    assert _attend(sinks=-1) == bad
    assert _attend(out=_fake([10, 8, 128], B.F16)) == bad                 # neither q's type nor f32
    assert _attend(out=_fake([9, 8, 128], B.BF16)) == bad
    assert _attend(q=_fake([10, 8, 128], B.I32), out=_fake([10, 8, 128], B.I32)) == bad
    assert _attend(q=_fake([10, 8, 128], B.BF16, strides=[2048, 256, 2])) == bad
    assert _attend(out=_fake([10, 8, 128], B.BF16, strides=[0, 128, 1])) == bad      # rows of out overlap
    assert _attend(out=_fake([10, 8, 128], B.BF16, strides=[1024, 0, 1])) == bad
    assert _attend(out=_fake([10, 8, 128], B.BF16, strides=[512, 128, 1])) == bad
    assert _attend(starts=_fake([2], B.I32)) == bad                       # B + 1 entries
    assert _attend(starts=_fake([3], B.I64)) == bad
    assert _attend(lens=_fake([3], B.I32)) == bad
    assert _attend(table=_fake([2, 4], B.I64)) == bad
    assert _attend(table=_fake([2, 4], B.I32, strides=[2, 1])) == bad     # rows overlap
    assert _attend(pages=_fake([4, 16, 2, 128], B.U8)) == bad             # slot too small
    assert _attend(pages=_fake([4, 16, 2, 140], B.U8)) == bad             # not a multiple of 8
    assert _attend(pages=_fake([4, 16, 2, 136], B.U8, ptr=0x10004)) == bad
    assert _attend(pages=_fake([4, 16, 2, 136], B.U8, strides=[4356, 272, 136, 1])) == bad
    assert _attend(pages=_fake([4, 16, 3, 136], B.U8)) == bad             # 8 query heads over 3
    assert _attend(pages=_fake([4, 8, 2, 136], B.U8)) == no               # block size
    assert _attend(cb=_books(B, kb=5), pages=_fake([4, 16, 2, 160], B.U8)) == no
    q96 = _fake([10, 8, 96], B.BF16)
    assert _attend(q=q96, out=q96, cb=_books(B, d=96)) == no
    many = _fake([1 << 20, 8, 128], B.BF16)
    assert _attend(q=many, out=many, max_q=1 << 20) == no                 # row tiles past the grid


def test_attend_of_nothing():
    B, _ = _lib()
    none = _fake([0, 8, 128], B.BF16, strides=[1024, 128, 1], ptr=0)
    assert _attend(q=none, out=none) == B.OK
    assert _attend(q=none, out=none, starts=_fake([1], B.I32), table=_fake([0, 4], B.I32, strides=[4, 1], ptr=0),
                   lens=_fake([0], B.I32, strides=[1], ptr=0)) == B.OK


def test_decode_window_refusals():
    B, lib = _lib()
    q = _fake([2, 8, 128], B.BF16)

    def dec(window=4, sinks=0, q=q, lens=_fake([2], B.I32)):
        return lib.tq_paged_decode_window(q, q, _fake([4, 16, 2, 136], B.U8), _fake([2, 4], B.I32), lens,
                                          ctypes.byref(_books(B)), 0, 0.1, window, sinks, None)

    assert dec(window=0) == B.ERR_INVALID_ARG
    assert dec(window=-3) == B.ERR_INVALID_ARG
    assert dec(sinks=-1) == B.ERR_INVALID_ARG
    assert dec(q=_fake([3, 8, 128], B.BF16)) == B.ERR_INVALID_ARG
    assert dec(lens=_fake([2], B.I64)) == B.ERR_INVALID_ARG


def _layers(B, *t):
    return (B.TensorDesc * len(t))(*t), len(t)


def _resize(**kw):
    B, lib = _lib()
    a = dict(layers=_layers(B, _fake([4, 16, 2, 136], B.U8)), table=_fake([2, 4], B.I32), lens=_fake([2], B.I32),
             new=_fake([2], B.I32), refs=_fake([4], B.I32), moves=_fake([2, 2], B.I32), window=0, sinks=0)
    a.update(kw)
    return lib.tq_pages_resize(a["layers"][0], a["layers"][1], a["table"], a["lens"], a["new"], a["refs"], a["moves"],
                               a["window"], a["sinks"], None)


def test_resize_refusals():
    B, _ = _lib()
    bad, no = B.ERR_INVALID_ARG, B.ERR_UNSUPPORTED
    page = lambda *s, **k: _fake(list(s), B.U8, **k)                       # noqa: E731
    assert _resize(layers=(None, 1)) == bad
    assert _resize(layers=_layers(B, page(4, 16, 2, 136))[:1] + (0,)) == bad
    assert _resize(layers=_layers(B, *[page(4, 16, 2, 136)] * 129)) == no
    assert _resize(layers=_layers(B, page(4, 16, 2, 136), page(5, 16, 2, 136))) == bad    # other page counts
    assert _resize(layers=_layers(B, page(4, 8, 2, 136))) == no
    assert _resize(layers=_layers(B, page(4, 16, 2, 132))) == bad
    assert _resize(layers=_layers(B, page(4, 16, 2, 136, ptr=0x10008))) == bad
    assert _resize(layers=_layers(B, page(4, 16, 2, 136, strides=[4352, 136, 2176, 1]))) == bad
    assert _resize(layers=_layers(B, page(4, 16, 2, 136, strides=[2176, 272, 136, 1]))) == bad   # overlap
    assert _resize(refs=_fake([5], B.I32)) == bad
    assert _resize(refs=_fake([4], B.I64)) == bad
    assert _resize(new=_fake([3], B.I32)) == bad
    assert _resize(moves=_fake([2, 3], B.I32)) == bad
    assert _resize(moves=_fake([2, 2], B.I32, strides=[4, 1])) == bad
    assert _resize(window=-1) == bad
    assert _resize(sinks=-1) == bad
    big = (1 << 21) + 1
    assert _resize(layers=_layers(B, page(big, 16, 2, 136)), refs=_fake([big], B.I32)) == no
    n = 8193
    assert _resize(table=_fake([n, 4], B.I32), lens=_fake([n], B.I32), new=_fake([n], B.I32),
                   moves=_fake([n, 2], B.I32)) == no
    none = _fake([0], B.I32, strides=[1], ptr=0)
    assert _resize(table=_fake([0, 4], B.I32, strides=[4, 1], ptr=0), lens=none, new=none,
                   moves=_fake([0, 2], B.I32, strides=[2, 1], ptr=0)) == B.OK


def test_fork_and_compact_refusals():
    B, lib = _lib()
    one, n = _layers(B, _fake([4, 16, 2, 136], B.U8))
    table, lens, refs = _fake([2, 4], B.I32), _fake([2], B.I32), _fake([4], B.I32)

    def fork(parents=_fake([1], B.I32), children=_fake([1], B.I32), moves=_fake([1, 2], B.I32)):
        return lib.tq_pages_fork(one, n, table, lens, refs, parents, children, moves, None)

    assert fork(children=_fake([2], B.I32)) == B.ERR_INVALID_ARG
    assert fork(parents=_fake([1], B.I64)) == B.ERR_INVALID_ARG
    assert fork(moves=_fake([2, 2], B.I32)) == B.ERR_INVALID_ARG
    none = _fake([0], B.I32, strides=[1], ptr=0)
    assert fork(none, none, _fake([0, 2], B.I32, strides=[2, 1], ptr=0)) == B.OK

    def compact(pos=_fake([2, 9], B.I32), counts=_fake([2], B.I32), dst=_fake([2, 1], B.I32), lens=lens):
        return lib.tq_pages_compact(one, n, table, lens, pos, counts, dst, None)

    assert compact(pos=_fake([3, 9], B.I32)) == B.ERR_INVALID_ARG
    assert compact(pos=_fake([2, 9], B.I64)) == B.ERR_INVALID_ARG
    assert compact(counts=_fake([1], B.I32)) == B.ERR_INVALID_ARG
    assert compact(dst=_fake([3, 1], B.I32)) == B.ERR_INVALID_ARG
    assert compact(lens=_fake([1], B.I32)) == B.ERR_INVALID_ARG
    assert compact(pos=_fake([2, 0], B.I32, strides=[1, 1], ptr=0)) == B.OK


def test_binding_refuses_cpu_tensors():
    import kv_cache_vector_append_b200 as tq
    z = torch.zeros(1, dtype=torch.int32)
    pages = torch.zeros(4, 16, 2, 136, dtype=torch.uint8)
    with pytest.raises(ValueError):
        tq.pages_resize(pages, z[None], z, z, z, z[None])
    with pytest.raises(ValueError):
        tq.pages_fork([pages, pages], z[None], z, z, z, z, z[None])
    with pytest.raises(ValueError):
        tq.pages_compact([], z[None], z, z[None], z, z[None])
