"""Arguments that the Python layer refuses before the library sees them (no GPU needed)."""
import pytest
import torch

import kv_cache_vector_append_b200 as tq


@pytest.mark.parametrize("name", ["max_q", "window", "sinks"])
@pytest.mark.parametrize("n", [2**31, 2**32 + 5, 2**63 - 1, -2**31 - 1])
def test_numbers_past_32_bits(name, n):
    """2^32 + 5 would arrive as 5."""
    z = torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 2, 128)
    pages = torch.zeros(4, 16, 2, 136, dtype=torch.uint8)
    numbers = dict(max_q=1, window=4, sinks=1)
    numbers[name] = n
    match = f"{name}={n}"
    with pytest.raises(ValueError, match=match):
        tq.paged_attend(q, q, z, pages, z[None], z, None, 0, 1.0, **numbers)
    if name != "max_q":
        del numbers["max_q"]
        with pytest.raises(ValueError, match=match):
            tq.paged_decode_window(q, q, pages, z[None], z, None, 0, 1.0, **numbers)
        with pytest.raises(ValueError, match=match):
            tq.pages_resize(pages, z[None], z, z, z, z[None], **numbers)
