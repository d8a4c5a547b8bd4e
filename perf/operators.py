"""Workloads of the paged-cache operators: growing block tables, storing K/V
rows in the pool, attention over whole prompts and attention of new rows over
the paged cache.

Each case is one call of one of them, in its plain form (elementary torch
operations) or, with ``own`` true, through the library's binding. ``exact``
states the same results in 64 bits, from the definitions.

A request's way through them: ``spec_extend_paged`` gives it blocks and maps
its rows to pool slots, ``spec_attend_prompt`` attends its prompt,
``spec_store_kv`` puts the prompt's K/V rows into the pool, and in every round
``spec_attend_paged`` attends the drafted rows over the cache before the check
and the commit.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # One sequence takes one more token: the engine's smallest step, all latency.
        dict(name="extend-1", kind="extend", B=1, bs=16, ctx_lo=511, ctx_hi=511, add_lo=1,
             add_hi=1, pad=0, lens_seed=1),
        # An engine round: 256 sequences of 128-2048 tokens grow by up to 5 (K + 1 rows).
        dict(name="extend-round-256", kind="extend", B=256, bs=16, ctx_lo=128, ctx_hi=2048,
             add_lo=0, add_hi=5, pad=64, lens_seed=2),
        # A whole batch of prompts is admitted: 64 requests of 512-4096 tokens.
        dict(name="extend-admit-64", kind="extend", B=64, bs=16, ctx_lo=0, ctx_hi=0, add_lo=512,
             add_hi=4096, pad=1000, lens_seed=3),
        # One round's new rows of 64 decoding sequences, one layer (8 heads of 128).
        dict(name="store-64", kind="store", T=64, heads=8, dim=128, layers=2, layer=1, bs=16,
             dtype="bf16", pad=0),
        # The packed K/V rows of a batch of prompts, with padding rows behind the last.
        dict(name="store-20000", kind="store", T=20000, heads=8, dim=128, layers=2, layer=0,
             bs=16, dtype="bf16", pad=77),
        # One short prompt of a small model: the smallest prompt call.
        dict(name="prompt-97-d64-fp16", kind="prompt", B=1, len_lo=97, len_hi=97, q_heads=16,
             kv_heads=2, dim=64, dtype="fp16", lens_seed=4),
        # A batch of packed prompts of very different lengths.
        dict(name="prompt-16-ragged", kind="prompt", B=16, len_lo=33, len_hi=2047, q_heads=32,
             kv_heads=8, dim=128, dtype="bf16", lens_seed=5),
        # One long prompt.
        dict(name="prompt-8192", kind="prompt", B=1, len_lo=8192, len_hi=8192, q_heads=32,
             kv_heads=8, dim=128, dtype="bf16", lens_seed=6),
        # One sequence decodes one token over a short cache: latency.
        dict(name="decode-1x700", kind="paged", B=1, ctx_lo=700, ctx_hi=700, n_lo=1, n_hi=1,
             staged=False, q_heads=32, kv_heads=8, dim=128, dtype="bf16", bs=16, layers=2,
             layer=1, lens_seed=7),
        # One sequence decodes one token over a long cache: a single row, split over the GPU.
        dict(name="decode-1x65000", kind="paged", B=1, ctx_lo=65000, ctx_hi=65000, n_lo=1,
             n_hi=1, staged=False, q_heads=32, kv_heads=8, dim=128, dtype="fp16", bs=16,
             layers=1, layer=0, lens_seed=8),
        # The rows of one chain check before it: 64 sequences, K + 1 = 9 rows each, whose own
        # K/V rows still lie in the commit's staging buffer; contexts 512-4096, blocks of 16.
        dict(name="verify-64x9-staged", kind="paged", B=64, ctx_lo=512, ctx_hi=4096, n_lo=9,
             n_hi=9, staged=True, q_heads=32, kv_heads=8, dim=128, dtype="bf16", bs=16, layers=2,
             layer=1, lens_seed=9),
        # Prompt chunks of different lengths over what is already cached of the prompt.
        dict(name="chunk-4x512", kind="paged", B=4, ctx_lo=4000, ctx_hi=8192, n_lo=300, n_hi=512,
             staged=False, q_heads=32, kv_heads=8, dim=128, dtype="bf16", bs=16, layers=2,
             layer=0, lens_seed=10),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    """One more case: sizes spread over the listed ones' ranges by their logarithm."""
    kind = rng.choice(["extend", "store", "prompt", "paged", "paged", "prompt"])
    seed = rng.randrange(1 << 30)
    if kind == "extend":
        B = _log_int(rng, 1, 512)
        hi = _log_int(rng, 1, min(4096, 260000 // B))
        ctx = rng.choice([0, 1]) * _log_int(rng, 1, 4096)
        return dict(kind=kind, B=B, bs=rng.choice([8, 16, 16, 32, 24]), ctx_lo=ctx // 2,
                    ctx_hi=ctx, add_lo=rng.randint(0, hi), add_hi=hi, pad=rng.randint(0, 500),
                    lens_seed=seed)
    dim = rng.choice([64, 128, 128, 96, 80])
    kv = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if kind == "store":
        layers = rng.choice([1, 2, 3])
        return dict(kind=kind, T=_log_int(rng, 1, 20000), heads=kv, dim=dim, layers=layers,
                    layer=rng.randrange(layers), bs=rng.choice([8, 16, 16, 32, 24]), dtype=dtype,
                    pad=rng.randint(0, 40))
    group = rng.choice([1, 2, 4, 4, 8, 3, 7])
    group = min(group, 32 // kv)
    if kind == "prompt":
        hi = _log_int(rng, 1, 8192)
        most = max(1, min(32, int(8192 * 8192 * 32 * 0.9) // (hi * hi * kv * group)))
        B = _log_int(rng, 1, most)
        return dict(kind=kind, B=B, len_lo=max(1, hi // rng.choice([1, 2, 20])), len_hi=hi,
                    q_heads=kv * group, kv_heads=kv, dim=dim, dtype=dtype, lens_seed=seed)
    n = _log_int(rng, 1, 512)
    staged = n <= 32 and rng.random() < 0.5
    ctx = max(n + 1, _log_int(rng, 1, 65000 if n <= 16 else 8192))
    most = max(1, min(64, 64 * 4096 * 8 // (ctx * kv), 4 * 512 * 32 * 8000 // (n * kv * group * ctx)))
    B = _log_int(rng, 1, most)
    layers = rng.choice([1, 2])
    return dict(kind=kind, B=B, ctx_lo=max(n + 1, ctx // rng.choice([1, 4])), ctx_hi=ctx,
                n_lo=n if staged else rng.randint(1, n), n_hi=n, staged=staged,
                q_heads=kv * group, kv_heads=kv, dim=dim, dtype=dtype,
                bs=rng.choice([8, 16, 16, 32, 64]), layers=layers, layer=rng.randrange(layers),
                lens_seed=seed)


def _lens(seed, count, lo, hi):
    r = random.Random(seed)
    return [r.randint(lo, hi) for _ in range(count)]


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(shape, gen, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(DTYPES[dtype])


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _blocks(n, bs):
    return -(-n // bs)


def _dealt_tables(lens, bs, max_blocks, num_blocks, seed):
    """Block tables of the given lengths with ids dealt at random (a pool in
    use for a while), the other ids on the free stack in random order."""
    ids = np.random.default_rng(seed).permutation(num_blocks).astype(np.int32)
    tables = np.full((len(lens), max_blocks), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        nb = _blocks(n, bs)
        tables[b, :nb] = ids[at:at + nb]
        at += nb
    stack = np.full(num_blocks, -1, np.int32)
    stack[:num_blocks - at] = ids[at:]
    return (torch.from_numpy(tables).cuda(), torch.from_numpy(stack).cuda(),
            _ints([num_blocks - at]))


def prepare(case, seed):
    return {"extend": _prepare_extend, "store": _prepare_store, "prompt": _prepare_prompt,
            "paged": _prepare_paged}[case["kind"]](case, seed)


def _prepare_extend(c, seed):
    lens = _lens(c["lens_seed"], c["B"], c["ctx_lo"], c["ctx_hi"])
    add = _lens(c["lens_seed"] + 1, c["B"], c["add_lo"], c["add_hi"])
    bs = c["bs"]
    max_blocks = max(_blocks(a + n, bs) for a, n in zip(lens, add)) + 2
    need = sum(_blocks(a + n, bs) for a, n in zip(lens, add))
    tables, stack, top = _dealt_tables(lens, bs, max_blocks, need + 32, seed)
    cap = sum(add) + c["pad"]
    return dict(kind="extend", bs=bs, tables=tables, lens=_ints(lens), add=_ints(add),
                stack=stack, top=top, status=_ints([0]),
                new_lens=torch.empty(c["B"], dtype=torch.int32, device="cuda"),
                new_top=torch.empty(1, dtype=torch.int32, device="cuda"),
                row_off=torch.empty(c["B"] + 1, dtype=torch.int32, device="cuda"),
                slot_map=torch.empty(cap, dtype=torch.int64, device="cuda"))


def _prepare_store(c, seed):
    g = _gen(seed)
    bs, T = c["bs"], c["T"]
    num_blocks = _blocks(T, bs) + 8
    pool = _rand((num_blocks, c["layers"], 2, bs, c["heads"], c["dim"]), g, c["dtype"])
    # K and V as a model's projection leaves them: two parts of one row.
    kv = _rand((T + c["pad"], 2, c["heads"], c["dim"]), g, c["dtype"])
    blocks = torch.randperm(num_blocks, generator=g, device="cuda")[:_blocks(T, bs)]
    pos = torch.arange(T, device="cuda")
    slots = torch.full((T + c["pad"],), -1, dtype=torch.int64, device="cuda")
    slots[:T] = blocks[pos // bs] * bs + pos % bs
    return dict(kind="store", k=kv[:, 0], v=kv[:, 1], slots=slots, rows=T, pool=pool,
                layer=c["layer"], bs=bs, status=_ints([0]))


def _offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).tolist()


def _prepare_prompt(c, seed):
    g = _gen(seed)
    lens = _lens(c["lens_seed"], c["B"], c["len_lo"], c["len_hi"])
    T, D = sum(lens), c["dim"]
    q = _rand((T, c["q_heads"], D), g, c["dtype"], 2.0)
    k = _rand((T, c["kv_heads"], D), g, c["dtype"])
    v = _rand((T, c["kv_heads"], D), g, c["dtype"])
    return dict(kind="prompt", q=q, k=k, v=v, off=_ints(_offsets(lens)), longest=max(lens),
                scale=D ** -0.5, status=_ints([0]), out=torch.empty_like(q),
                lse=torch.empty((T, c["q_heads"]), dtype=torch.float32, device="cuda"))


def _paged_lens(c):
    ctx = _lens(c["lens_seed"], c["B"], c["ctx_lo"], c["ctx_hi"])
    n = _lens(c["lens_seed"] + 1, c["B"], c["n_lo"], c["n_hi"])
    return ctx, n


def _prepare_paged(c, seed):
    g = _gen(seed)
    ctx, n = _paged_lens(c)
    bs, D, T = c["bs"], c["dim"], sum(n)
    need = sum(_blocks(x, bs) for x in ctx)
    max_blocks = max(_blocks(x, bs) for x in ctx) + 1
    tables, _, _ = _dealt_tables(ctx, bs, max_blocks, need + 8, seed)
    pool = _rand((need + 8, c["layers"], 2, bs, c["kv_heads"], D), g, c["dtype"])
    stage = None
    if c["staged"]:
        stage = _rand((c["B"], c["n_hi"], c["layers"], 2, c["kv_heads"], D), g, c["dtype"])
    q = _rand((T, c["q_heads"], D), g, c["dtype"], 2.0)
    return dict(kind="paged", q=q, pool=pool, stage=stage, layer=c["layer"], tables=tables,
                lens=_ints(ctx), off=_ints(_offsets(n)), longest=max(ctx), most=max(n),
                scale=D ** -0.5, status=_ints([0]), out=torch.empty_like(q),
                lse=torch.empty((T, c["q_heads"]), dtype=torch.float32, device="cuda"))


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------
_kept = {}


def _workspace(capi, q):
    """The attention workspace a program keeps between its calls: one for each
    device and stream, as calls that may overlap need one each."""
    key = (q.get_device(), capi._stream(None), q.shape[-1])
    if key not in _kept:
        _kept[key] = capi.attend_workspace(q.shape[-1], device=q.device)
    return _kept[key]


def run(s):
    if own:
        return _run_own(s)
    return {"extend": _plain_extend, "store": _plain_store, "prompt": _plain_prompt,
            "paged": _plain_paged}[s["kind"]](s)


def _run_own(s):
    from speculative_decoding_verification_89_b200 import capi
    if s["kind"] == "extend":
        capi.spec_extend_paged(s["tables"], s["lens"], s["add"], s["stack"], s["top"],
                               s["new_lens"], s["new_top"], s["row_off"], s["status"],
                               block_size=s["bs"], slot_map=s["slot_map"])
        return dict(tables=s["tables"], lens=s["new_lens"], top=s["new_top"],
                    row_off=s["row_off"], slots=s["slot_map"])
    if s["kind"] == "store":
        capi.spec_store_kv(s["k"], s["v"], s["slots"], s["pool"], s["layer"], s["status"])
        return s["pool"]
    ws = _workspace(capi, s["q"])
    if s["kind"] == "prompt":
        capi.spec_attend_prompt(s["q"], s["k"], s["v"], s["off"], s["out"], s["status"], ws,
                                scale=s["scale"], lse=s["lse"])
    else:
        capi.spec_attend_paged(s["q"], s["pool"], s["layer"], s["tables"], s["lens"], s["out"],
                               s["status"], ws, row_off=s["off"], kv_stage=s["stage"],
                               scale=s["scale"], lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"])


def _plain_extend(s):
    bs, lens, add = s["bs"], s["lens"], s["add"]
    new = lens + add
    held, need = (lens + bs - 1) // bs, (new + bs - 1) // bs
    miss = need - held
    before = torch.cumsum(miss, 0) - miss
    col = torch.arange(s["tables"].shape[1], device="cuda")
    fresh = (col >= held[:, None]) & (col < need[:, None])
    pop = (s["top"] - 1 - (before[:, None] + col - held[:, None])).clamp(0, len(s["stack"]) - 1)
    tables = torch.where(fresh, s["stack"][pop], s["tables"])
    off = torch.zeros(len(lens) + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.cumsum(add, 0)
    row = torch.arange(len(s["slot_map"]), device="cuda")
    b = torch.searchsorted(off[1:], row, right=True).clamp(max=len(lens) - 1)
    pos = (lens[b] + row - off[b]).clamp(0, tables.shape[1] * bs - 1)
    slots = tables[b, pos // bs].long() * bs + pos % bs
    return dict(tables=tables, lens=new, top=(s["top"] - miss.sum()).to(torch.int32), row_off=off,
                slots=torch.where(row < off[-1], slots, -1))


def _plain_store(s):
    at = s["slots"][:s["rows"]]
    block, row = at // s["bs"], at % s["bs"]
    s["pool"][:, s["layer"], 0][block, row] = s["k"][:s["rows"]]
    s["pool"][:, s["layer"], 1][block, row] = s["v"][:s["rows"]]
    return s["pool"]


def _padded(x, off, most):
    """Packed rows [T, H, D] as [B, H, most, D] in 32 bits (what follows a
    sequence's end is not used)."""
    at = (off[:-1, None] + torch.arange(most, device="cuda")).clamp(max=x.shape[0] - 1)
    return x[at].float().transpose(1, 2)


def _plain_attend(q, k, v, seen, scale, off, T, dtype):
    """q [B, Hq, R, D], k and v [B, Hkv, L, D], seen [B or 1, R, L]: packed
    rows of the attention and its log-sum-exp."""
    B, Hq, R, D = q.shape
    Hkv, L = k.shape[1], k.shape[2]
    w = torch.matmul(q.reshape(B, Hkv, Hq // Hkv * R, D), k.transpose(2, 3)).mul_(scale)
    w = w.view(B, Hkv, Hq // Hkv, R, L).masked_fill_(~seen[:, None, None], float("-inf"))
    top = w.amax(-1, keepdim=True)
    w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(B, Hkv, Hq // Hkv * R, L), v).view(B, Hq, R, D)
    o = o / total.view(B, Hq, R, 1)
    lse = (top + total.log()).view(B, Hq, R)
    row = torch.arange(T, device="cuda")
    b = torch.searchsorted(off[1:], row, right=True)
    at = row - off[b]
    return dict(out=o[b, :, at].to(dtype), lse=lse[b, :, at].contiguous())


def _plain_prompt(s):
    q, k, v = (_padded(s[x], s["off"], s["longest"]) for x in "qkv")
    at = torch.arange(s["longest"], device="cuda")
    return _plain_attend(q, k, v, (at <= at[:, None])[None], s["scale"], s["off"],
                         s["q"].shape[0], s["q"].dtype)


def _plain_paged(s):
    pool, bs = s["pool"][:, s["layer"]], s["pool"].shape[3]
    table = s["tables"][:, :_blocks(s["longest"], bs)].clamp(min=0)
    k, v = (pool[:, i][table].flatten(1, 2).float().transpose(1, 2) for i in (0, 1))
    q = _padded(s["q"], s["off"], s["most"])
    key = torch.arange(k.shape[2], device="cuda")
    row = torch.arange(s["most"], device="cuda")
    if s["stage"] is None:
        first = s["lens"] - (s["off"][1:] - s["off"][:-1])
        seen = key <= (first[:, None] + row)[:, :, None]
    else:
        st = s["stage"][:, :s["most"], s["layer"]].float()
        k = torch.cat([k, st[:, :, 0].transpose(1, 2)], 2)
        v = torch.cat([v, st[:, :, 1].transpose(1, 2)], 2)
        cached = (key < s["lens"][:, None])[:, None].expand(-1, len(row), -1)
        fresh = (row <= row[:, None])[None].expand(len(s["lens"]), -1, -1)
        seen = torch.cat([cached, fresh], 2)
    return _plain_attend(q, k, v, seen, s["scale"], s["off"], s["q"].shape[0], s["q"].dtype)


# ----------------------------------------------------------------------------
# What one pass cannot do without
# ----------------------------------------------------------------------------
def work(c):
    if c["kind"] == "extend":
        lens = _lens(c["lens_seed"], c["B"], c["ctx_lo"], c["ctx_hi"])
        add = _lens(c["lens_seed"] + 1, c["B"], c["add_lo"], c["add_hi"])
        held = sum(_blocks(x, c["bs"]) for x in lens)
        fresh = sum(_blocks(x + a, c["bs"]) for x, a in zip(lens, add)) - held
        # lengths, counts, the entry of each sequence's last block and popped
        # ids read; new entries, lengths, offsets and slots written
        return dict(bytes=20 * c["B"] + 8 * fresh + 8 * (sum(add) + c["pad"]), flops=0)
    if c["kind"] == "store":
        return dict(bytes=c["T"] * (8 * c["heads"] * c["dim"] + 8), flops=0)
    Hq, Hkv, D = c["q_heads"], c["kv_heads"], c["dim"]
    if c["kind"] == "prompt":
        lens = _lens(c["lens_seed"], c["B"], c["len_lo"], c["len_hi"])
        pairs, keys, rows = sum(n * (n + 1) // 2 for n in lens), sum(lens), sum(lens)
    else:
        ctx, n = _paged_lens(c)
        first = ctx if c["staged"] else [x - m for x, m in zip(ctx, n)]
        pairs = sum(f * m + m * (m + 1) // 2 for f, m in zip(first, n))
        keys, rows = sum(f + m for f, m in zip(first, n)), sum(n)
    return dict(bytes=4 * D * (keys * Hkv + rows * Hq) + 4 * rows * Hq, flops=4 * D * Hq * pairs)


# ----------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    """Attention one sequence and one head at a time; a store is a copy, and
    growing tables gives whole numbers only."""
    if case["kind"] == "extend":
        return None
    s = prepare(case, seed)
    if case["kind"] == "store":
        pool = s["pool"].double()
        for part, rows in enumerate((s["k"], s["v"])):
            flat = pool[:, s["layer"], part].flatten(0, 1)
            flat[s["slots"][:s["rows"]]] = rows[:s["rows"]].double()
            pool[:, s["layer"], part] = flat.view_as(pool[:, s["layer"], part])
        return pool
    T, Hq, D = s["q"].shape
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, Hq), dtype=torch.float64, device="cuda")
    off = s["off"].tolist()
    for b in range(len(off) - 1):
        rows = slice(off[b], off[b + 1])
        n = off[b + 1] - off[b]
        if case["kind"] == "prompt":
            keys, values = s["k"][rows], s["v"][rows]
        else:
            length, bs = int(s["lens"][b]), s["pool"].shape[3]
            ids = s["tables"][b, :_blocks(length, bs)].long()
            cached = s["pool"][ids, s["layer"]]
            keys = cached[:, 0].reshape(-1, *cached.shape[3:])[:length]
            values = cached[:, 1].reshape(-1, *cached.shape[3:])[:length]
            if s["stage"] is not None:
                keys = torch.cat([keys, s["stage"][b, :n, s["layer"], 0]])
                values = torch.cat([values, s["stage"][b, :n, s["layer"], 1]])
        L = keys.shape[0]
        hidden = torch.ones((n, L), dtype=torch.bool, device="cuda").triu(L - n + 1)
        group = Hq // keys.shape[1]
        for h in range(Hq):
            scores = s["q"][rows, h].double() @ keys[:, h // group].double().T * s["scale"]
            scores[hidden] = -math.inf
            z = torch.logsumexp(scores, dim=1)
            lse[rows, h] = z
            out[rows, h] = torch.exp(scores - z[:, None]) @ values[:, h // group].double()
    return dict(out=out, lse=lse)
