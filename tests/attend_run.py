"""Helpers of the paged-cache and attention tests: inputs, the CUDA path and
the oracle's results with a derived error bound."""
from __future__ import annotations

import numpy as np
import torch

from oracle.attend import attend_rows, cached_rows

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def rand(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))


def deal_tables(lens, bs, num_blocks, max_blocks, seed):
    """Tables with ids dealt at random; entries past a sequence's blocks hold
    ids that must not be read (the largest int)."""
    ids = np.random.default_rng(seed).permutation(num_blocks)
    t = np.full((len(lens), max_blocks), np.iinfo(np.int32).max, np.int32)
    at = 0
    for b, n in enumerate(lens):
        nb = -(-n // bs)
        t[b, :nb] = ids[at:at + nb]
        at += nb
    assert at <= num_blocks
    return torch.from_numpy(t)


def check(out, lse, want, dtype, D):
    """Compares one sequence's rows with the oracle's. The bound, per element:
    each weight is rounded once to dtype (half a step u of it, or 2^-25 where
    fp16 is subnormal, weights being relative to at least 1), the result once
    (u); the scores are fp32 sums of D products (error at most (D + 4) 2^-24 of
    the sum of their absolute values), and scaling, exponentials and the sums
    over keys add less than 2^-18 relative."""
    u = HALF_STEP[dtype]
    score = (D + 4) * 2.0 ** -24 * want.qk
    g = 2 * score + 2.0 ** -18 + 2.0 ** -22 * want.qk
    tol = (u + g[..., None]) * want.mass * 1.01 + u * np.abs(want.out) * 1.01
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25 * want.vsum + 2.0 ** -25
    o = f64(out)
    bad = ~(np.abs(o - want.out) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(o - want.out).max(), tol[bad][:4])
    if lse is not None:
        z = f64(lse)
        empty = np.isneginf(want.lse)
        assert (np.isneginf(z) == empty).all()
        ok = np.abs(z - want.lse) <= g + 2.0 ** -22 * np.abs(want.lse)
        assert (ok | empty).all(), (z[~ok], want.lse[~ok])


def check_prompt(q, k, v, lens, out, lse, scale):
    at = 0
    for n in lens:
        r = slice(at, at + n)
        want = attend_rows(f64(q[r]), f64(k[r]), f64(v[r]), scale)
        check(out[r], None if lse is None else lse[r], want, q.dtype, q.shape[-1])
        at += n


def check_paged(q, pool, layer, tables, lens, rows, out, lse, scale, stage=None):
    p, at = f64(pool[:, layer]), 0
    for b, n in enumerate(rows):
        r = slice(at, at + n)
        k, v = cached_rows(p, tables[b].tolist(), int(lens[b]))
        if stage is not None:
            k = np.concatenate([k, f64(stage[b, :n, layer, 0])])
            v = np.concatenate([v, f64(stage[b, :n, layer, 1])])
        want = attend_rows(f64(q[r]), k, v, scale)
        check(out[r], None if lse is None else lse[r], want, q.dtype, q.shape[-1])
        at += n
