"""Plain 64-bit forms of the attention over chunks and windows and of the page operations."""
import numpy as np
import torch

from oracle import tq_oracle as O
from tests.gpu_helpers import oracle_table

BS = 16


def attend_ref(q, starts, pages, table, lens, d, kb, vb, seed, scale, window=0, sinks=0, out_eps=0.0,
               num_blocks=None):
    """(out, tol): the definition row by row in float64, and the largest 2-norm of a row's error.

    Each fp16 rounding is 2^-11 off at most.  A score is scale nK <q', c>; q', c, nK and c nK are
    rounded, q' and c per coordinate with random signs: the sum over D coordinates of products of
    two unit vectors that the rotation has spread (sum of their squared products about 1/D, 3/D at
    most) is off by sigma <= scale |q| |k| 2^-11 sqrt(4/3) sqrt(3/D), of which 6 sigma are taken; the
    rounding of nK scales the score.  A value weight is rounded four times (weight, c, nV, c nV).  So
    |error| <= sum_t p_t |v_t| (2 delta_s + 4 * 2^-11), plus the rounding of the output.
    """
    q = np.asarray(q, dtype=np.float64)
    hq, hkv = q.shape[1], pages.shape[2]
    g = hq // hkv
    kt, vt = oracle_table(d, kb), oracle_table(d, vb)
    kreg, vreg = O.region_bytes(d, kb), O.region_bytes(d, vb)
    signs = O.rht_signs(d, seed)
    nb = pages.shape[0] if num_blocks is None else num_blocks
    out = np.zeros_like(q)
    tol = np.zeros(q.shape[:2])
    u = 2.0 ** -11
    for b in range(len(lens)):
        n = int(lens[b])
        nq = int(starts[b + 1] - starts[b])
        if n == 0 or nq == 0:
            continue
        t = np.arange(n)
        ids = np.asarray(table[b])[t // BS]
        there = (ids >= 0) & (ids < nb)
        slots = pages[np.where(there, ids, 0), t % BS]                     # [n, H_kv, stride]
        ki, kn = O.decode_region(slots[..., :kreg], d, kb)
        vi, vn = O.decode_region(slots[..., kreg:kreg + vreg], d, vb)
        bad = ~(np.isfinite(kn) & np.isfinite(vn))
        khat = O.dequantize_rows(ki, np.where(bad, 0, kn), kt, signs)
        vhat = O.dequantize_rows(vi, np.where(bad, 0, vn), vt, signs)
        kl, vl = np.linalg.norm(khat, axis=-1), np.linalg.norm(vhat, axis=-1)
        for i in range(nq):
            p = n - nq + i
            see = there & (t <= p)
            if window > 0:
                see &= (t > p - window) | (t < sinks)
            if not see.any():
                continue
            for h in range(hq):
                kv, row = h // g, starts[b] + i
                s = scale * (khat[see, kv] @ q[row, h])
                w = np.exp(s - s.max())
                w /= w.sum()
                out[row, h] = w @ vhat[see, kv]
                if bad[see, kv].any():
                    out[row, h] = np.nan
                ds = abs(scale) * np.linalg.norm(q[row, h]) * kl[see, kv].max() * u * 6 * 2 / np.sqrt(d) + \
                    np.abs(s).max() * u
                tol[row, h] = (w @ vl[see, kv]) * (2 * ds + 4 * u) + out_eps * np.linalg.norm(out[row, h])
    return out, tol


def check_rows(got, ref, tol, out_eps=None):
    """NaN exactly where the reference is; elsewhere every row within its tolerance (+ a denormal).

    With out_eps also all rows together, within out_eps + 4e-3 of their 2-norm: over many rows the
    roundings of a score count with their variance, scale |q| |k| 2^-11 / sqrt(3) sqrt(2 / D) with
    |k| <= 100 for the keys of these tests and scale |q| about 1, at most 3.6e-3 (D = 64; that of
    the weights' error, whose mean drops out, is no larger), and those of values and weights
    2^-11 each.
    """
    nan = np.isnan(ref).any(-1)
    assert np.array_equal(np.isnan(got).any(-1), nan)
    err = np.linalg.norm(np.where(nan[..., None], 0, got - ref), axis=-1)
    tol = np.where(nan, 0, tol)
    worst = np.max(err / (tol + 1e-30)) if err.size else 0.0
    assert np.all(err <= tol + 1e-7), (worst, np.argwhere(err > tol + 1e-7)[:5])
    if out_eps is not None:
        rel = np.linalg.norm(err) / max(np.linalg.norm(np.where(nan[..., None], 0, ref)), 1e-30)
        assert rel <= out_eps + 4e-3, rel
    return worst


def out_eps(dtype):
    return torch.finfo(dtype).eps / 2


# ---- page operations, request by request -------------------------------------------------------

def pages_of(n):
    return (n + BS - 1) // BS


def resize_ref(pages, table, lens, new, refs, window=0, sinks=0):
    """In place on numpy arrays (pages: a list); returns moves."""
    cols, pool = table.shape[1], len(refs)
    free = [i for i in range(pool) if refs[i] == 0]
    start = refs.copy()
    asked, plan = 0, []
    for b in range(len(lens)):
        n, m = int(lens[b]), int(new[b])
        if not (0 <= n <= cols * BS and 0 <= m <= cols * BS):
            plan.append(None)
            continue
        last = table[b, n // BS] if n % BS else -1
        copy = bool(m > n and n % BS and 0 <= last < pool and start[last] > 1)
        need = max(0, pages_of(m) - pages_of(n)) + copy
        first, asked = asked, asked + need
        plan.append((first, need, copy) if need == 0 or asked <= len(free) else None)
    moves = np.full((len(lens), 2), -1, np.int32)
    for b, what in enumerate(plan):
        if what is None:
            moves[b] = -2
            continue
        first, need, copy = what
        n, m = int(lens[b]), int(new[b])
        got = free[first:first + need]
        for p in got:
            refs[p] = 1
        if copy:
            old = table[b, n // BS]
            moves[b] = (old, got[0])
            table[b, n // BS] = got[0]
            refs[old] -= 1
            got = got[1:]
        table[b, pages_of(n):pages_of(n) + len(got)] = got
        for c in range(pages_of(n)):
            gone = c >= pages_of(m)
            if window > 0 and c * BS >= sinks and (c + 1) * BS <= min(n, m) - window + 1:
                gone = True
            if gone:
                if 0 <= table[b, c] < pool:
                    refs[table[b, c]] -= 1
                table[b, c] = -1
        lens[b] = m
    for old, new_page in moves[moves[:, 0] >= 0]:
        for p in pages:
            p[new_page] = p[old]
    return moves


def fork_ref(pages, table, lens, refs, parents, children):
    nb, cols, pool = len(lens), table.shape[1], len(refs)
    free = [i for i in range(pool) if refs[i] == 0]
    at_start = lens.copy()
    asked, named = 0, set()
    moves = np.full((len(parents), 2), -1, np.int32)
    for i, (a, c) in enumerate(zip(parents, children)):
        first_name = c not in named
        if 0 <= c < nb:
            named.add(c)
        ok = 0 <= a < nb and 0 <= c < nb and first_name and at_start[c] == 0 and \
            0 <= at_start[a] <= cols * BS
        if not ok:
            moves[i] = -2
            continue
        n = int(at_start[a])
        tail = table[a, n // BS] if n % BS else -1
        need = int(0 <= tail < pool)
        asked += need
        if need and asked > len(free):
            moves[i] = -2
            continue
        for col in range(n // BS if need else pages_of(n)):
            table[c, col] = table[a, col]
            if 0 <= table[a, col] < pool:
                refs[table[a, col]] += 1
        if need:
            moves[i] = (tail, free[asked - 1])
            table[c, n // BS] = free[asked - 1]
            refs[free[asked - 1]] = 1
        lens[c] = n
    for old, new_page in moves[moves[:, 0] >= 0]:
        for p in pages:
            p[new_page] = p[old]
    return moves


def compact_ref(pages, table, lens, pos, counts, dst):
    pool = pages[0].shape[0]
    for p in pages:
        before = p.copy()
        for b in range(len(lens)):
            if not (0 <= counts[b] <= min(pos.shape[1], dst.shape[1] * BS)) or \
                    not 0 <= lens[b] <= table.shape[1] * BS:
                continue
            for i in range(counts[b]):
                t = pos[b, i]
                if not 0 <= t < lens[b]:
                    continue
                src, to = table[b, t // BS], dst[b, i // BS]
                if 0 <= src < pool and 0 <= to < pool:
                    p[to, i % BS] = before[src, t % BS]
