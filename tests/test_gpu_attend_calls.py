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
