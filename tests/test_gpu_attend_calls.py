"""Calls of tq_paged_attend and tq_paged_decode_window that the documentation allows at the ends of
their ranges."""
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
