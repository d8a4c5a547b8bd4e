"""Plain attention over packed or paged keys, block-table growth and K/V store
(the oracle).

TEST INFRASTRUCTURE ONLY: no product code imports it, and it shares no code
with the CUDA path.

HiSpec (gist.science summary of arXiv 2510.01336), section 2
"Unterstuetzung fuer Batch-Inferenz" names paged attention with block tables
and prints no formula; the formula here is the usual one. Row i of a
sequence's n new rows sees its first L - n + i + 1 of L keys.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

STATUS_OK, STATUS_EINVAL, STATUS_ENOBLOCKS = 0, -1, -4


@dataclass
class AttendResult:
    out: np.ndarray    # [n, Hq, D] float64
    lse: np.ndarray    # [n, Hq] natural log of the sum of exponentials, -inf for an empty row
    mass: np.ndarray   # [n, Hq, D] sum_j p_j |v_j|
    vsum: np.ndarray   # [n, Hq, D] sum_j |v_j| over the keys seen
    qk: np.ndarray     # [n, Hq] max_j sum_d |q_d k_jd| * scale over the keys seen


def attend_rows(q, k, v, scale) -> AttendResult:
    """q [n, Hq, D], k and v [L, Hkv, D] (float64): see the module."""
    n, Hq, D = q.shape
    L, Hkv = k.shape[:2]
    g = Hq // Hkv
    out = np.zeros((n, Hq, D))
    mass, vsum = np.zeros_like(out), np.zeros_like(out)
    lse = np.full((n, Hq), -np.inf)
    qk = np.zeros((n, Hq))
    for i in range(n):
        seen = min(L, max(0, L - n + i + 1))
        if seen == 0:
            continue
        for h in range(Hq):
            kk, vv = k[:seen, h // g], v[:seen, h // g]
            s = kk @ q[i, h] * scale
            m = s.max()
            e = np.exp(s - m)
            tot = e.sum()
            out[i, h] = e @ vv / tot
            lse[i, h] = m + np.log(tot)
            mass[i, h] = e @ np.abs(vv) / tot
            vsum[i, h] = np.abs(vv).sum(0)
            qk[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
    return AttendResult(out, lse, mass, vsum, qk)


def cached_rows(pool, table, length):
    """K and V rows 0..length-1 [length, H, D] of one sequence from one layer's
    pool [num_blocks, 2, block_size, H, D]."""
    bs = pool.shape[2]
    k = np.array([pool[table[p // bs], 0, p % bs] for p in range(length)])
    v = np.array([pool[table[p // bs], 1, p % bs] for p in range(length)])
    shape = (length,) + pool.shape[3:]
    return k.reshape(shape), v.reshape(shape)


@dataclass
class ExtendResult:
    status: int
    tables: np.ndarray
    lens: np.ndarray
    free_top: int
    row_off: np.ndarray
    slots: np.ndarray


def extend_paged(tables, seq_lens, add_len, free_stack, free_top, block_size, num_blocks,
                 capacity) -> ExtendResult:
    """Grow sequences one after the other, one row at a time, taking a block
    from the top of the stack whenever a row starts one."""
    tables = np.array(tables, dtype=np.int64, copy=True)
    B, max_blocks = tables.shape
    lens = np.array(seq_lens, dtype=np.int64, copy=True)
    add = np.asarray(add_len, dtype=np.int64)
    off = np.zeros(B + 1, np.int64)
    slots = np.full(capacity, -1, np.int64)

    def fail(code):
        return ExtendResult(code, np.array(tables_in), np.array(seq_lens), int(free_top), off,
                            slots)
    tables_in = np.array(tables, copy=True)
    if (lens < 0).any() or (add < 0).any() or not 0 <= free_top <= num_blocks:
        return fail(STATUS_EINVAL)
    if ((lens + add + block_size - 1) // block_size > max_blocks).any() or add.sum() > capacity:
        return fail(STATUS_EINVAL)
    for b in range(B):
        if add[b] and lens[b] % block_size and \
                not 0 <= tables[b, lens[b] // block_size] < num_blocks:
            return fail(STATUS_EINVAL)
    missing = int(((lens + add + block_size - 1) // block_size
                   - (lens + block_size - 1) // block_size).sum())
    if missing > free_top:
        return fail(STATUS_ENOBLOCKS)
    top, row = int(free_top), 0
    for b in range(B):
        off[b] = row
        for _ in range(add[b]):
            pos = lens[b]
            if pos % block_size == 0:
                top -= 1
                if not 0 <= free_stack[top] < num_blocks:
                    return fail(STATUS_EINVAL)
                tables[b, pos // block_size] = free_stack[top]
            slots[row] = tables[b, pos // block_size] * block_size + pos % block_size
            lens[b] += 1
            row += 1
    off[B] = row
    return ExtendResult(STATUS_OK, tables, lens, top, off, slots)
