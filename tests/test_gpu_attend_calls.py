"""Calls of tq_paged_attend and tq_paged_decode_window that the documentation allows at the ends of
their ranges."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests.attend_helpers import check_rows
from tests.gpu_helpers import to_np_f64
from tests.test_gpu_attend import SEED, Case, _tq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
def test_max_q_of_zero_leaves_every_new_token_out(d):
    tq = _tq()
    c = Case(tq, d, 4, 2, 4, 4, [60, 0, 33], [1, 0, 3])
    c.max_q = 0
    c.run()
    assert tq.get_device_error() == tq.DEVERR_SEQLEN_RANGE
    assert torch.all(c.out == 7.0)
    c.starts.fill_(2)                                        # no sequence has new tokens
    c.run()
    assert tq.get_device_error() == 0
    assert torch.all(c.out == 7.0)


def test_a_prompt_of_131072_tokens_in_one_call():
    """524,288 query rows of one KV head, through a window; rows checked one by one."""
    tq = _tq()
    n, window, sinks = 131072, 16, 2
    c = Case(tq, 64, 4, 1, 2, 2, [n], [n])
    got = to_np_f64(c.run(window, sinks))
    assert tq.get_device_error() == 0
    q, lens, starts = c.q, c.lens, c.starts
    rng = np.random.default_rng(0)
    for p in [0, 1, 15, 16, 17, 255, 256, n - 257, n - 2, n - 1] + rng.integers(0, n, 20).tolist():
        # row p alone, of the sequence up to it
        first = max(0, (p - window) // 16 * 16)
        keep = np.r_[0:16, first:p + 1] if first > 16 else np.arange(p + 1)
        c.q = q[p:p + 1]
        c.lens, c.starts = lens * 0 + len(keep), starts * 0 + torch.tensor([0, 1], device="cuda", dtype=torch.int32)
        table = c.table
        c.table = table[:, torch.as_tensor(keep[::16] // 16, device="cuda").long()]
        check_rows(got[p:p + 1], *c.ref(window, sinks))
        c.table = table


FIRST_USE = """
import torch
import kv_cache_vector_append_b200 as tq
from tests.test_gpu_attend import Case, SEED
cases = [Case(tq, d, 4, 2, kb, vb, [300, 77], q) for d, kb, vb, q in
         ((128, 4, 4, [1, 1]), (64, 3, 8, [90, 40]), (128, 8, 2, [70, 30]), (256, 2, 3, [40, 60]), (256, 3, 3, [2, 1]))]
cases[0].run()                                              # the library's first attention, outside a capture
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
pages = torch.zeros(30, 16, 2, 136, dtype=torch.uint8, device="cuda")
table, lens, refs, moves, new = i32([[-1] * 4] * 3), i32([0] * 3), i32([0] * 30), i32([[0, 0]] * 3), i32([20, 17, 0])
parents, children, pos, counts = i32([0]), i32([2]), i32([[5, 3]]), i32([2])
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for c in cases[1:]:
        c.run(50, 3)
    tq.pages_resize(pages, table, lens, new, refs, moves)
    tq.pages_fork(pages, table, lens, refs, parents, children, moves[:1])
    tq.pages_compact(pages, table[:1], lens[:1], pos, counts, table[1:2])
graph.replay()
torch.cuda.synchronize()
assert lens.tolist() == [20, 17, 20] and refs.sum().item() == 6, (lens, refs)
for c in cases[1:]:
    got = c.out.clone()
    c.out.fill_(7.0)
    assert torch.equal(c.run(50, 3), got)
assert tq.get_device_error() == 0
"""


def test_kernels_first_used_inside_a_capture():
    """Only the library's first call on a device has to come before a capture: every other kernel may
    be loaded inside one."""
    _tq()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_USE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("d,q_lens", [(128, [1, 2]), (64, [4, 3]), (128, [90, 40]), (256, [40, 70])])
def test_out_may_be_q(d, q_lens):
    """Every block reads its queries before any row of theirs is written."""
    tq = _tq()
    c = Case(tq, d, 8, 2, 4, 4, [2300, 100], q_lens)
    want = c.run().clone()
    c.out = c.q
    assert torch.equal(c.run(), want)
