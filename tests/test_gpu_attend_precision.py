"""How far tq_paged_attend may be from the definition, all rows together, where the roundings of its
fp16 operands are amplified or hidden: keys that share a direction (channel means)."""
import numpy as np
import pytest
import torch

from oracle import tq_oracle as O
from tests.attend_helpers import BS
from tests.gpu_helpers import oracle_table, to_np_f64
from tests.test_gpu_attend import SEED, Case, _tq

pytestmark = pytest.mark.gpu
HALF_STEP = 2.0 ** -11                      # fp16


def _mean_keys(tq, c, mean, seed=3):
    """c's pages with keys N(mean_d, 1), the channel means N(0, mean^2) and the same for all heads,
    and values N(0, 1)."""
    s = c.spec
    g = torch.Generator().manual_seed(seed)
    lens = c.lens.tolist()
    table = c.table.cpu().numpy()
    slots = np.concatenate([table[b, np.arange(n) // BS].astype(np.int64) * BS + np.arange(n) % BS
                            for b, n in enumerate(lens)])
    mu = torch.randn(s.head_dim, generator=g) * mean
    k = torch.randn(len(slots), s.num_kv_heads, s.head_dim, generator=g) + mu
    v = torch.randn(len(slots), s.num_kv_heads, s.head_dim, generator=g)
    tq.quantize_append(c.pages, torch.from_numpy(slots).cuda(), k.cuda(), v.cuda(), c.cb, SEED)


def _factor_residual(cents):
    """Mean squared rounding of fp16 centroids under the best of the factors 1 + j / 512."""
    best = None
    for j in range(512):
        a = np.float32(1 + j / 512)
        r = (cents * a).astype(np.float16).astype(np.float64) / a - cents
        if best is None or (r ** 2).mean() < (best ** 2).mean():
            best = r
    return best


def _definition(c):
    """(out, relative error allowed) of all rows: a row of a whole sequence sees all up to its own.

    A rounding to fp16 is off by 2^-11 relative at most, by 2^-11 / sqrt 3 in the mean square; those
    of weights, value centroids and their products with the norms are independent of each other and
    move the output by that much each.  Score errors move it by their own size.  The query's, per
    coordinate, cost scale |q| |k - mean k| / sqrt D times that: what all keys share drops out of the
    softmax.  What a key centroid is off by, e (8 bits: nothing, hi + lo), costs scale |q| |k| e.  The
    squares add.  1.25: the mean over a few hundred rows.
    """
    s = c.spec
    d, hkv, g = s.head_dim, s.num_kv_heads, s.num_q_heads // s.num_kv_heads
    kt, vt = oracle_table(d, s.k_bits), oracle_table(d, s.v_bits)
    kreg, vreg = O.region_bytes(d, s.k_bits), O.region_bytes(d, s.v_bits)
    signs = O.rht_signs(d, SEED)
    pages, table, starts = c.pages.cpu().numpy(), c.table.cpu().numpy(), c.starts.cpu().numpy()
    q = to_np_f64(c.q)
    out, var = np.zeros_like(q), 0.0
    residual = np.zeros(1 << s.k_bits) if s.k_bits == 8 else _factor_residual(np.asarray(kt.centroids, np.float64))
    for b, n in enumerate(c.lens.tolist()):
        nq = int(starts[b + 1] - starts[b])
        t = np.arange(n)
        slot = pages[table[b][t // BS], t % BS]
        ki, kn = O.decode_region(slot[..., :kreg], d, s.k_bits)
        vi, vn = O.decode_region(slot[..., kreg:kreg + vreg], d, s.v_bits)
        khat, vhat = O.dequantize_rows(ki, kn, kt, signs), O.dequantize_rows(vi, vn, vt, signs)
        hide = t[None, :] > (n - nq + np.arange(nq))[:, None]
        for h in range(s.num_q_heads):
            x = c.scale * (q[starts[b]:starts[b + 1], h] @ khat[:, h // g].T)
            x[hide] = -np.inf
            w = np.exp(x - x.max(-1, keepdims=True))
            out[starts[b]:starts[b + 1], h] = w @ vhat[:, h // g] / w.sum(-1, keepdims=True)
        ql2 = c.scale ** 2 * (q[starts[b]:starts[b + 1]] ** 2).sum(-1).mean()
        spread = ((khat - khat.mean(0)) ** 2).sum(-1).mean()
        e2 = (np.asarray(kn, np.float64) ** 2).mean() * (residual[ki] ** 2).mean()
        var = max(var, ql2 * (spread / d * HALF_STEP ** 2 / 3 + e2))
    return out, 1.25 * np.sqrt(3 * HALF_STEP ** 2 / 3 + var)


def _check_mean_keys(d, hq, hkv, kb, vb, lens, q_lens, mean):
    tq = _tq()
    c = Case(tq, d, hq, hkv, kb, vb, lens, q_lens, "f32")
    _mean_keys(tq, c, mean)
    ref, allowed = _definition(c)
    err = np.linalg.norm(to_np_f64(c.run()) - ref) / np.linalg.norm(ref)
    assert err <= allowed, (err, allowed)
    assert tq.get_device_error() == 0


@pytest.mark.parametrize("mean", [0, 10, 30])
@pytest.mark.parametrize("d,vb,lens,q_lens", [(64, 8, [700, 90], [100, 90]), (128, 4, [700, 90], [33, 90]),
                                              (128, 8, [1500], [40]), (256, 2, [700, 50], [70, 50]),
                                              (256, 8, [1500], [40])])
def test_8_bit_keys_that_share_a_direction_in_chunks(d, vb, lens, q_lens, mean):
    _check_mean_keys(d, 4, 2, 8, vb, lens, q_lens, mean)


@pytest.mark.parametrize("mean", [0, 10, 30])
@pytest.mark.parametrize("d,kb,vb,q_len", [(256, 3, 4, 12), (256, 4, 2, 16), (128, 4, 4, 4), (128, 3, 8, 14),
                                           (64, 4, 3, 16), (64, 2, 4, 8), (128, 8, 4, 16), (256, 8, 8, 16),
                                           (256, 3, 4, 40), (128, 4, 4, 40), (64, 4, 3, 80)])
def test_keys_that_share_a_direction(d, kb, vb, q_len, mean):
    _check_mean_keys(d, 4, 2, kb, vb, [300, 417, 333, 512, 100], [q_len] * 5, mean)


@pytest.mark.parametrize("kb", [2, 3, 4, 8])
@pytest.mark.parametrize("vb", [2, 3, 4, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [12, 40])
def test_every_width_pair_together(d, kb, vb, q_len):
    _check_mean_keys(d, 4, 2, kb, vb, [200, 317, 133, 61], [q_len] * 4, 1)


@pytest.mark.parametrize("d,hq,hkv,kb,vb,q_lens", [(128, 8, 2, 4, 4, [8, 5]), (128, 8, 2, 4, 2, [100, 41]),
                                                   (64, 14, 2, 8, 8, [4, 4]), (64, 14, 2, 8, 8, [60, 20]),
                                                   (256, 4, 2, 3, 4, [16, 9]), (256, 4, 2, 4, 3, [50, 70])])
def test_long_sequences_together(d, hq, hkv, kb, vb, q_lens):
    _check_mean_keys(d, hq, hkv, kb, vb, [5001, 2100], q_lens, 3)
