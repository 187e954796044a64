"""Cases for the operators of a packed-KV server: attention of a chunk of new tokens over the
packed pages, single-token attention with a sliding window and sinks, and the page operations
(resize, fork, compact), with a plain torch form of each and an exact one in 64 bits.

A slot holds one (token, KV head): [K codes | fp32 norm | V codes | fp32 norm]; a key is
nK R^T cK[code], a value nV R^T cV[code], R = (1/sqrt D) H diag(s) the seeded Hadamard rotation.
"""

import math
import os
import struct

import numpy as np
import torch

own = False

BS = 16                    # tokens per page
SIGN_SEED = 0x5EED
CODEBOOKS = os.path.join("kv_cache_vector_append_b200", "codebooks")

# (head_dim, query heads, KV heads, K bits, V bits): the layers of the bench's workloads, and one
# with 256-wide heads
QWEN05 = dict(d=64, hq=14, hkv=2, kb=8, vb=8)
LLAMA = dict(d=128, hq=32, hkv=8, kb=4, vb=4)
QWEN7 = dict(d=128, hq=28, hkv=4, kb=4, vb=2)
LONG = dict(d=128, hq=32, hkv=8, kb=3, vb=2)
WIDE = dict(d=256, hq=16, hkv=4, kb=4, vb=4)
LAYERS = (QWEN05, LLAMA, QWEN7, LONG, WIDE)


def listed():
    return [
        # speculative verification: a few draft tokens of eight sequences
        dict(name="attend verify 4 tokens", op="attend", **QWEN05, batch=8, chunk=4, ctx=4096, ragged=True,
             window=0, sinks=0, dtype="bfloat16"),
        # chunked prefill of a mixed batch
        dict(name="attend chunk 512", op="attend", **LLAMA, batch=4, chunk=512, ctx=8192, ragged=True,
             window=0, sinks=0, dtype="bfloat16"),
        # one long prompt, a late chunk of it
        dict(name="attend long prompt", op="attend", **LONG, batch=1, chunk=4096, ctx=20480, ragged=False,
             window=0, sinks=0, dtype="bfloat16"),
        # a prompt chunk of a model with a sliding window, sink tokens kept
        dict(name="attend window", op="attend", **QWEN7, batch=3, chunk=1999, ctx=12000, ragged=True,
             window=4096, sinks=4, dtype="float16"),
        # one user, one new token: latency
        dict(name="decode window 1 user", op="decode", **LLAMA, batch=1, ctx=20000, ragged=False,
             window=1024, sinks=4, dtype="bfloat16"),
        # a full decode batch of ragged sequences
        dict(name="decode window batch", op="decode", **QWEN7, batch=64, ctx=32768, ragged=True,
             window=4096, sinks=4, dtype="bfloat16"),
        # a decode step of a small batch: at most one new page a sequence
        dict(name="resize one token", op="resize", **LLAMA, batch=8, ctx=2000, grow=1, pool=4096, window=0,
             sinks=0),
        # a big pool: prompts of up to 4096 tokens admitted at once, then released
        dict(name="resize admit prompts", op="resize", **QWEN05, batch=256, ctx=2048, grow=4096, pool=131072,
             window=0, sinks=0),
        # several answers to one prompt
        dict(name="fork 8 samples", op="fork", **LLAMA, parents=1, children=8, ctx=1000, layers=4),
        # a step of a beam search over many prompts
        dict(name="fork beams", op="fork", **QWEN7, parents=32, children=128, ctx=8192, layers=4),
        # one short sequence cut to its kept tokens
        dict(name="compact one", op="compact", **QWEN7, batch=1, ctx=1000, keep=257, layers=1),
        # a batch cut to a quarter of its tokens
        dict(name="compact batch", op="compact", **LLAMA, batch=16, ctx=32768, keep=8191, layers=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attend", "attend", "decode", "resize", "fork", "compact"))
    layer = dict(rng.choice(LAYERS))
    if op == "attend":
        window = rng.choice((0, 0, _log(rng, 64, 8192)))
        chunk = _log(rng, 1, 2048)
        return dict(op=op, **layer, batch=_log(rng, 1, 8), chunk=chunk, ctx=chunk + _log(rng, 1, 12000),
                    ragged=rng.random() < 0.7, window=window, sinks=rng.choice((0, 1, 4, 16)) if window else 0,
                    dtype=rng.choice(("bfloat16", "float16")))
    if op == "decode":
        return dict(op=op, **layer, batch=_log(rng, 1, 64), ctx=_log(rng, 1, 32768), ragged=rng.random() < 0.7,
                    window=_log(rng, 1, 8192), sinks=rng.choice((0, 1, 4, 64)),
                    dtype=rng.choice(("bfloat16", "float16")))
    if op == "resize":
        window = rng.choice((0, 0, _log(rng, 64, 2048)))
        batch, ctx, grow = _log(rng, 1, 256), _log(rng, 1, 2048), _log(rng, 1, 4096)
        return dict(op=op, **QWEN05, batch=batch, ctx=ctx, grow=grow,
                    pool=min(131072, batch * ((ctx + grow) // BS + 2) + _log(rng, 1, 65536)), window=window,
                    sinks=rng.choice((0, 4)) if window else 0)
    if op == "fork":
        parents = _log(rng, 1, 32)
        return dict(op=op, **layer, parents=parents, children=parents * _log(rng, 1, 4), ctx=_log(rng, 1, 8192),
                    layers=_log(rng, 1, 4))
    ctx = _log(rng, 16, 16384)
    return dict(op=op, **layer, batch=_log(rng, 1, 16), ctx=ctx, keep=max(1, int(ctx * rng.uniform(0.05, 0.9))),
                layers=_log(rng, 1, 2))


# ---- inputs ----------------------------------------------------------------------------------

def _slot_bytes(c):
    return c["d"] * c["kb"] // 8 + 4 + c["d"] * c["vb"] // 8 + 4


def _table(d, bits):
    with open(os.path.join(CODEBOOKS, "beta_d%d_b%d.tqcb" % (d, bits)), "rb") as f:
        raw = f.read()
    n = 1 << bits
    return (torch.tensor(struct.unpack_from("<%df" % n, raw, 32)),
            torch.tensor(struct.unpack_from("<%df" % (n - 1), raw, 32 + 4 * n)))


def _signs(d):
    """s_j = -1 where bit 63 of the j-th SplitMix64 output is set."""
    out, m = [], (1 << 64) - 1
    for j in range(d):
        z = (SIGN_SEED + (j + 1) * 0x9E3779B97F4A7C15) & m
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & m
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & m
        out.append(-1.0 if (z ^ (z >> 31)) >> 63 else 1.0)
    return torch.tensor(out, dtype=torch.float64)


def _rotation(d):
    i = np.arange(d)
    h = np.array([bin(x).count("1") & 1 for x in (i[:, None] & i[None, :]).reshape(-1)]).reshape(d, d)
    return torch.from_numpy(1.0 - 2.0 * h) / math.sqrt(d) * _signs(d)[None, :]


def _pack(codes, bits):
    """codes [N, D] -> little-endian bit stream [N, D bits / 8]."""
    n, d = codes.shape
    b = (codes.unsqueeze(-1) >> torch.arange(bits, device=codes.device)) & 1
    b = b.reshape(n, d * bits // 8, 8)
    return (b << torch.arange(8, device=codes.device)).sum(-1).to(torch.uint8)


def _geometry(case):
    """Lengths belong to the case: a generator that is the same for every seed."""
    return torch.Generator().manual_seed(case["ctx"] * 1009 + case.get("batch", 0))


def _lengths(case, hi, lo):
    """Sequence lengths: all `hi`, or spread over [lo, hi] with the longest among them."""
    n, g = case["batch"], _geometry(case)
    if not case["ragged"]:
        return torch.full((n,), hi, dtype=torch.int64)
    t = torch.randint(lo, hi + 1, (n,), generator=g)
    t[0] = hi
    return t


def _fill(case, blocks, gpu):
    """A pool of quantized rows: keys with log-normal channel scales and two outlier channels,
    Gaussian values, rotated, their unit coordinates coded by the Lloyd-Max cells."""
    d, hkv = case["d"], case["hkv"]
    sigma = torch.exp(0.5 * torch.randn(hkv, d, device="cuda", generator=gpu))
    sigma[:, :2] *= 20.0
    rot = _rotation(d).to("cuda", torch.float32)
    pages = torch.empty(blocks, BS, hkv, _slot_bytes(case), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 18) // (BS * hkv))
    for p in range(0, blocks, step):
        n = min(step, blocks - p)
        parts = []
        for bits, scale in ((case["kb"], sigma), (case["vb"], 1.0)):
            x = torch.randn(n, BS, hkv, d, device="cuda", generator=gpu) * scale
            norm = x.norm(dim=-1, keepdim=True)
            u = (x @ rot.t()) / norm
            codes = torch.bucketize(u, _table(d, bits)[1].cuda()).reshape(-1, d)
            parts += [_pack(codes, bits), norm.reshape(-1, 1).view(torch.uint8).reshape(-1, 4)]
        pages[p:p + n] = torch.cat(parts, dim=-1).reshape(n, BS, hkv, -1)
    return pages


def _i32(t):
    return t.to(torch.int32).cuda()


def _fork_rows(case):
    """Parents' lengths, and the parent of each child: the children go round the parents."""
    g = _geometry(case)
    lens = torch.randint((case["ctx"] + 1) // 2, case["ctx"] + 1, (case["parents"],), generator=g)
    lens[0] = case["ctx"]
    return lens, torch.arange(case["children"]) % case["parents"]


def prepare(case, seed):
    op = case["op"]
    g = torch.Generator().manual_seed(seed)
    gpu = torch.Generator("cuda").manual_seed(seed)
    s = dict(case=case)
    if op in ("attend", "decode"):
        dtype = getattr(torch, case["dtype"])
        lens = _lengths(case, case["ctx"], max(1, case["ctx"] // 8))
        nblk = (lens + BS - 1) // BS
        pool = int(nblk.sum()) + 3
        order = torch.randperm(pool, generator=g)
        bt = torch.full((case["batch"], int(nblk.max())), -1, dtype=torch.int64)
        at = 0
        for b in range(case["batch"]):
            bt[b, :nblk[b]] = order[at:at + nblk[b]]
            at += int(nblk[b])
        s.update(pages=_fill(case, pool, gpu), table=_i32(bt), lens=_i32(lens), host_lens=lens.tolist(),
                 scale=1.0 / math.sqrt(case["d"]))
        if op == "attend":
            ql = torch.minimum(_lengths(case, case["chunk"], max(1, case["chunk"] // 2)), lens)
            starts = torch.cat([torch.zeros(1, dtype=torch.int64), ql.cumsum(0)])
            s.update(starts=_i32(starts), host_starts=starts.tolist(), max_q=int(ql.max()))
            rows = int(starts[-1])
        else:
            rows = case["batch"]
        s["q"] = torch.randn(rows, case["hq"], case["d"], device="cuda", generator=gpu).to(dtype)
        s["out"] = torch.zeros_like(s["q"])
        s["rot"] = _rotation(case["d"]).to("cuda", torch.float32)
        s["kc"], s["vc"] = (_table(case["d"], case[k])[0].cuda() for k in ("kb", "vb"))
        if own:
            import kv_cache_vector_append_b200 as tq
            s["codebooks"] = tq.load_codebooks(case["d"], case["kb"], case["vb"], "cuda")
        return s
    if op == "compact":
        b, n = case["batch"], (case["ctx"] + BS - 1) // BS
        m = (case["keep"] + BS - 1) // BS
        order = torch.randperm(b * (n + m), generator=g)
        counts = torch.randint(max(1, case["keep"] // 2), case["keep"] + 1, (b,), generator=g)
        counts[0] = case["keep"]
        pos = torch.rand(b, case["ctx"], device="cuda", generator=gpu).argsort(dim=1)[:, :case["keep"]]
        first = torch.arange(case["keep"], device="cuda")[None, :] < counts.cuda()[:, None]
        pos = torch.where(first, pos, case["ctx"]).sort(dim=1).values
        s.update(pages=_random_pages(case, b * (n + m), gpu), table=_i32(order[:b * n].reshape(b, n)),
                 lens=_i32(torch.full((b,), case["ctx"])), pos=_i32(pos), counts=_i32(counts),
                 dst=_i32(order[b * n:].reshape(b, m)))
        return s
    if op == "resize":
        b = case["batch"]
        base = torch.randint(0, case["ctx"] + 1, (b,), generator=g)
        more = base + torch.randint(1, case["grow"] + 1, (b,), generator=g)
        cols = (case["ctx"] + case["grow"]) // BS + 2
        n = (base + BS - 1) // BS
        pool = case["pool"]
        s.update(base=_i32(base), more=_i32(more))
    else:
        plens, parent = _fork_rows(case)
        b = case["parents"] + case["children"]
        base = torch.cat([plens, torch.zeros(case["children"], dtype=torch.int64)])
        n = (base + BS - 1) // BS
        cols = int(n.max()) + 1
        pool = int(n.sum()) + 2 * case["children"]
        s.update(parent=_i32(parent), child=_i32(case["parents"] + torch.arange(case["children"])),
                 without=_i32(base))
    order = torch.randperm(pool, generator=g)
    col = torch.arange(cols)[None, :]
    used = col < n[:, None]
    table = torch.full((b, cols), -1, dtype=torch.int64)
    table[used] = order[:int(n.sum())]
    refs = torch.zeros(pool, dtype=torch.int64)
    refs[order[:int(n.sum())]] = 1
    s.update(table=_i32(table), lens=_i32(base), refs=_i32(refs), pages=_random_pages(case, pool, gpu),
             moves=torch.full((b if op == "resize" else case["children"], 2), -1, dtype=torch.int32, device="cuda"),
             moves_r=torch.full((b, 2), -1, dtype=torch.int32, device="cuda"))
    return s


def _random_pages(case, blocks, gpu):
    """Pools for the operators that move packed slots without reading into them."""
    shape = (blocks, BS, case["hkv"], _slot_bytes(case))
    return [torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=gpu)
            for _ in range(case.get("layers", 1))]


# ---- one pass --------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        import kv_cache_vector_append_b200 as tq
    if c["op"] == "attend":
        if own:
            tq.paged_attend(s["out"], s["q"], s["starts"], s["pages"], s["table"], s["lens"], s["codebooks"],
                            SIGN_SEED, s["scale"], s["max_q"], window=c["window"], sinks=c["sinks"])
            return s["out"]
        return _attend(s, s["host_starts"])
    if c["op"] == "decode":
        if own:
            tq.paged_decode_window(s["out"], s["q"], s["pages"], s["table"], s["lens"], s["codebooks"], SIGN_SEED,
                                   s["scale"], c["window"], sinks=c["sinks"])
            return s["out"]
        return _attend(s, list(range(c["batch"] + 1)))
    if c["op"] == "resize":
        # the sequences fall back to their short lengths, then grow
        for new in (s["base"], s["more"]):
            if own:
                tq.pages_resize(s["pages"], s["table"], s["lens"], new, s["refs"], s["moves"], window=c["window"],
                                sinks=c["sinks"])
            else:
                _resize(s["pages"], s["table"], s["lens"], new, s["refs"], s["moves"], c["window"], c["sinks"])
        return [s["table"], s["lens"], s["refs"], s["moves"]] + s["pages"]
    if c["op"] == "fork":
        # the children of the last step are released, then the parents fork again
        if own:
            tq.pages_resize(s["pages"], s["table"], s["lens"], s["without"], s["refs"], s["moves_r"])
            tq.pages_fork(s["pages"], s["table"], s["lens"], s["refs"], s["parent"], s["child"], s["moves"])
        else:
            _resize(s["pages"], s["table"], s["lens"], s["without"], s["refs"], s["moves_r"], 0, 0)
            _fork(s["pages"], s["table"], s["lens"], s["refs"], s["parent"], s["child"], s["moves"])
        return [s["table"], s["lens"], s["refs"], s["moves"]] + s["pages"]
    if own:
        tq.pages_compact(s["pages"], s["table"], s["lens"], s["pos"], s["counts"], s["dst"])
    else:
        _compact(s["pages"], s["table"], s["lens"], s["pos"], s["counts"], s["dst"])
    return s["pages"]


# ---- plain forms -----------------------------------------------------------------------------

def _dequant(rows, d, bits, off, cents):
    """[N, slot bytes] -> fp32 norm times centroid, [N, D] (rotated domain)."""
    p = torch.arange(d, device=rows.device) * bits
    reg = rows[:, off:off + d * bits // 8 + 4]
    w = reg[:, p // 8].to(torch.int32) | reg[:, p // 8 + 1].to(torch.int32) << 8
    norm = reg[:, d * bits // 8:].contiguous().view(torch.float32)
    return cents[((w >> (p % 8)) & ((1 << bits) - 1)).long()] * norm


def _attend(s, starts):
    c = s["case"]
    d, hq, hkv = c["d"], c["hq"], c["hkv"]
    grp, koff = hq // hkv, d * c["kb"] // 8 + 4
    out = torch.zeros_like(s["out"])
    for b, length in enumerate(s["host_lens"]):
        nq = starts[b + 1] - starts[b]
        ids = s["table"][b, :(length + BS - 1) // BS].long()
        rows = s["pages"][ids].reshape(-1, hkv, s["pages"].shape[-1])[:length].reshape(length * hkv, -1)
        k = (_dequant(rows, d, c["kb"], 0, s["kc"]) @ s["rot"]).reshape(length, hkv, d)
        v = (_dequant(rows, d, c["vb"], koff, s["vc"]) @ s["rot"]).reshape(length, hkv, d)
        q = s["q"][starts[b]:starts[b + 1]].float().reshape(nq, hkv, grp, d).permute(1, 0, 2, 3).reshape(hkv, -1, d)
        p = torch.arange(length - nq, length, device=q.device)[:, None]
        t = torch.arange(length, device=q.device)[None, :]
        see = t <= p
        if c["window"] > 0:
            see &= (t > p - c["window"]) | (t < c["sinks"])
        x = (q @ k.permute(1, 2, 0)).mul_(s["scale"]).reshape(hkv, nq, grp, length)
        x.masked_fill_(~see[None, :, None, :], -math.inf)
        top = x.amax(-1, keepdim=True)
        x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
        total = x.sum(-1, keepdim=True)
        o = x.reshape(hkv, nq * grp, length) @ v.permute(1, 0, 2)
        o = o.reshape(hkv, nq, grp, d) / torch.where(total == 0, torch.ones_like(total), total)
        out[starts[b]:starts[b + 1]] = o.permute(1, 0, 2, 3).reshape(nq, hq, d).to(out.dtype)
    return out


def _copy_pages(pages, moves):
    src, dst = moves[moves[:, 0] >= 0].long().unbind(1)
    for p in pages:
        p[dst] = p[src]


def _drop(refs, table, gone):
    """The table entries `gone` are released."""
    ids = torch.where(gone & (table >= 0), table, refs.numel()).long().reshape(-1)
    refs -= torch.bincount(ids, minlength=refs.numel() + 1)[:-1].to(refs.dtype)
    table.masked_fill_(gone, -1)


def _resize(pages, table, lens, new, refs, moves, window, sinks):
    b, cols = table.shape
    free = (refs == 0).nonzero().squeeze(1)
    have, want = (lens + BS - 1) // BS, (new + BS - 1) // BS
    last = table.gather(1, (have - 1).clamp(min=0).long()[:, None]).squeeze(1)
    shared = (new > lens) & (lens % BS != 0) & (last >= 0) & (refs[last.clamp(min=0).long()] > 1)
    need = (want - have).clamp(min=0) + shared
    end = need.cumsum(0)
    ok = (end <= free.numel()) | (need == 0)
    first = end - need
    page = lambda k: torch.cat([free, free.new_zeros(1)])[k.clamp(0, free.numel()).long()].to(torch.int32)  # noqa: E731
    col = torch.arange(cols, device=table.device, dtype=torch.int32)[None, :]
    least = torch.minimum(lens, new)
    gone = (col >= want[:, None]) & (col < have[:, None])
    if window > 0:
        gone |= (col < have[:, None]) & (col * BS >= sinks) & ((col + 1) * BS <= least[:, None] - window + 1)
    copy = ok & shared
    moves[:, 0] = torch.where(copy, last, -1)
    moves[:, 1] = torch.where(copy, page(first), -1)
    at_last = copy[:, None] & (col == have[:, None] - 1)
    refs -= torch.bincount(torch.where(copy, last, refs.numel()).long(), minlength=refs.numel() + 1)[:-1].int()
    table.copy_(torch.where(at_last, moves[:, 1:], table))
    grown = ok[:, None] & (col >= have[:, None]) & (col < want[:, None])
    table.copy_(torch.where(grown, page((first + shared)[:, None] + col - have[:, None]), table))
    refs[table[grown | at_last].long()] = 1
    _drop(refs, table, gone & ok[:, None])
    lens.copy_(torch.where(ok, new, lens))
    _copy_pages(pages, moves)


def _fork(pages, table, lens, refs, parent, child, moves):
    p, c = parent.long(), child.long()
    free = (refs == 0).nonzero().squeeze(1)
    full, part = lens[p] // BS, lens[p] % BS != 0
    tail = table[p].gather(1, full.clamp(max=table.shape[1] - 1).long()[:, None]).squeeze(1)
    need = (part & (tail >= 0)).int()
    end = need.cumsum(0)
    ok = (end <= free.numel()) | (need == 0)
    fresh = torch.cat([free, free.new_zeros(1)])[(end - need).clamp(max=free.numel()).long()].to(torch.int32)
    copy = ok & (need > 0)
    moves[:, 0] = torch.where(copy, tail, -1)
    moves[:, 1] = torch.where(copy, fresh, -1)
    col = torch.arange(table.shape[1], device=table.device, dtype=torch.int32)[None, :]
    share = ok[:, None] & (col < full[:, None])
    rows = torch.where(share, table[p], table[c])
    ids = torch.where(share & (rows >= 0), rows, refs.numel()).long().reshape(-1)
    refs += torch.bincount(ids, minlength=refs.numel() + 1)[:-1].to(refs.dtype)
    table[c] = torch.where(copy[:, None] & (col == full[:, None]), moves[:, 1:], rows)
    refs[moves[copy][:, 1].long()] = 1
    lens[c] = torch.where(ok, lens[p], lens[c])
    _copy_pages(pages, moves)


def _compact(pages, table, lens, pos, counts, dst):
    i = torch.arange(pos.shape[1], device=pos.device)[None, :]
    b, i = (i < counts[:, None]).nonzero().unbind(1)
    t = pos[b, i].long()
    src = table[b, t // BS].long() * BS + t % BS
    to = dst[b, i // BS].long() * BS + i % BS
    for p in pages:
        rows = p.view(-1, p.shape[2] * p.shape[3])
        rows[to] = rows[src]


# ---- work and exact values -------------------------------------------------------------------

def _visible(c, length, nq):
    """Visible (query, key) pairs, and the keys that some query sees."""
    p = np.arange(length - nq, length, dtype=np.int64)
    lo = np.maximum(0, p + 1 - c["window"]) if c["window"] > 0 else np.zeros_like(p)
    pairs = int((p + 1 - lo + np.minimum(lo, c["sinks"])).sum())
    return pairs, int(length - lo[0] + min(lo[0], c["sinks"]))


def work(case):
    """Bytes that have to be read or written and operations of one pass (lengths at their mean)."""
    d, op = case["d"], case["op"]
    slot = _slot_bytes(case)
    row = case["hkv"] * slot
    if op in ("attend", "decode"):
        size = case["batch"]
        mean = lambda hi, lo: hi if not case["ragged"] else (hi + lo) // 2  # noqa: E731
        length = mean(case["ctx"], max(1, case["ctx"] // 8))
        nq = min(length, mean(case["chunk"], max(1, case["chunk"] // 2))) if op == "attend" else 1
        pairs, keys = _visible(case, length, nq)
        return dict(bytes=size * (keys * row + 2 * nq * case["hq"] * d * 2 + 4 * ((keys + BS - 1) // BS) + 8),
                    flops=size * 4 * d * case["hq"] * pairs)
    if op == "resize":
        pages = case["batch"] * (case["grow"] // 2) // BS
        # both calls: the counts read, the entries and counts of the pages taken or released
        return dict(bytes=2 * (4 * case["pool"] + 12 * pages + 24 * case["batch"]), flops=0)
    if op == "fork":
        ctx = case["ctx"] * 3 // 4
        pool = case["parents"] * ctx // BS + 2 * case["children"]
        # release and fork: the shared entries and their counts, the last page of each child copied
        return dict(bytes=2 * 4 * pool + case["children"] * (2 * 16 * (ctx // BS) + 2 * case["layers"] * BS * row),
                    flops=0)
    kept = case["batch"] * (case["keep"] * 3 // 4)
    return dict(bytes=kept * (2 * case["layers"] * row + 4), flops=0)


def exact(case, seed):
    """The attention outputs in 64 bits: the queries rotated, scored on the codes, and the weighted
    centroids rotated back, one KV head at a time.  Page operations have whole outputs only."""
    if case["op"] not in ("attend", "decode"):
        return None
    s = prepare(case, seed)
    d, hkv, grp = case["d"], case["hkv"], case["hq"] // case["hkv"]
    rot = _rotation(d).cuda()
    koff = d * case["kb"] // 8 + 4
    starts = s["host_starts"] if case["op"] == "attend" else list(range(case["batch"] + 1))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    bit = torch.arange(8, device="cuda")
    for b, length in enumerate(s["host_lens"]):
        lo, hi = starts[b], starts[b + 1]
        at = torch.arange(length, device="cuda")
        flat = s["table"][b].long()[at // BS] * BS + at % BS
        p = length - (hi - lo) + torch.arange(hi - lo, device="cuda").repeat_interleave(grp)
        hide = at[None, :] > p[:, None]
        if case["window"] > 0:
            hide |= (at[None, :] <= p[:, None] - case["window"]) & (at[None, :] >= case["sinks"])
        for h in range(hkv):
            slots = s["pages"].reshape(-1, hkv, s["pages"].shape[-1])[flat, h]
            kv = []
            for off, bits, cents in ((0, case["kb"], s["kc"]), (koff, case["vb"], s["vc"])):
                n = d * bits // 8
                stream = ((slots[:, off:off + n, None].long() >> bit) & 1).reshape(length, d, bits)
                code = (stream << torch.arange(bits, device="cuda")).sum(-1)
                norm = slots[:, off + n:off + n + 4].contiguous().view(torch.float32).double()
                kv.append(cents.double()[code] * norm)
            q = s["q"][lo:hi, h * grp:(h + 1) * grp].double().reshape(-1, d) @ rot.T
            w = (q @ kv[0].T).mul_(s["scale"]).masked_fill_(hide, -math.inf)
            w = torch.softmax(w, dim=-1).nan_to_num_(0.0)
            o = (w @ kv[1]) @ rot
            out[lo:hi, h * grp:(h + 1) * grp] = o.reshape(hi - lo, grp, d)
    return out
