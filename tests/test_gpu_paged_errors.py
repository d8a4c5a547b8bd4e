"""Errors of the paged-cache and attention calls on the GPU: what a bad value
leaves done and undone, and what the next call finds."""
import numpy as np
import pytest
import torch

from oracle.attend import AttendResult, attend_rows
from tests.attend_run import check, f64, offsets, rand
from tests.test_gpu_attend import paged_inputs

pytestmark = pytest.mark.gpu


def _capi():
    from speculative_decoding_verification_89_b200 import capi
    return capi


def _status(code=0):
    return torch.full((1,), code, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("T", [1, 8, 9, 64, 65, 577, 20000])
@pytest.mark.parametrize("bad_at", ["first", "last", "both"])
def test_store_skips_bad_slots_only(T, bad_at):
    """A bad slot costs its own row and no other, however many rows the call
    has (more than run at once among them), and is flagged; a pending error
    stops the whole call, whatever the slots."""
    capi = _capi()
    bs, H, D = 16, 1, 64
    N = -(-T // bs) + 1
    pool = torch.zeros((N, 1, 2, bs, H, D), dtype=torch.bfloat16, device="cuda")
    kv = rand((T, 2, H, D), torch.bfloat16, T).cuda()
    slots = torch.randperm(N * bs, generator=torch.Generator().manual_seed(T))[:T].cuda()
    if bad_at != "last":
        slots[0] = N * bs
    if bad_at != "first":
        slots[-1] = -2
    want = pool.clone()
    ok = (slots >= 0) & (slots < N * bs)
    at = slots[ok]
    want[at // bs, 0, 0, at % bs], want[at // bs, 0, 1, at % bs] = kv[ok, 0], kv[ok, 1]
    for _ in range(3):
        pool.zero_()
        st = _status()
        capi.spec_store_kv(kv[:, 0], kv[:, 1], slots, pool, 0, st)
        torch.cuda.synchronize()
        assert int(st) == capi.SPEC_EINVAL and torch.equal(pool, want)
    pool.zero_()
    capi.spec_store_kv(kv[:, 0], kv[:, 1], slots, pool, 0, st)
    torch.cuda.synchronize()
    assert int(st) == capi.SPEC_EINVAL and not pool.any()
    capi.spec_store_kv(kv[:, 0], kv[:, 1], slots, pool, 0, None)   # no status word
    torch.cuda.synchronize()
    assert torch.equal(pool, want)


@pytest.mark.parametrize("lens,rows,heads,D,cta", [
    ([2500], [9], (4, 1), 128, 5), ([2500], [9], (4, 1), 128, 0),
    ([600, 1900, 40], [300, 1, 40], (8, 2), 128, 60), ([1500] * 60, [1] * 60, (4, 4), 64, 7),
])
@pytest.mark.parametrize("with_status", [True, False])
def test_attention_after_a_wait_that_ran_out(lens, rows, heads, D, cta, with_status):
    """One CTA's products never come, so its part of a divided unit is missing.
    The call ends, says so, and leaves the workspace ready: the next call, of
    other values, gives what it gives on a new workspace. (In the last case a
    unit's second part is written long before its first, so a count left over
    would join it too early.)"""
    capi = _capi()
    Hq, Hkv = heads
    pool, tables = paged_inputs(lens, 16, Hkv, D, torch.bfloat16, 20, layers=1)
    tables, off = tables.cuda(), offsets(rows).cuda()
    seq = torch.tensor(lens, dtype=torch.int32).cuda()
    ws = capi.attend_workspace(D)

    def call(seed, ws):
        q = rand((sum(rows), Hq, D), torch.bfloat16, seed, 2.0).cuda()
        out, lse, st = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda"), _status()
        capi.spec_attend_paged(q, pool, 0, tables, seq, out, st if with_status else None, ws,
                               row_off=off, lse=lse)
        torch.cuda.synchronize()
        return out, lse, int(st)

    assert capi._lib.spec_test_stop_attend_cta(cta) == capi.SPEC_OK
    try:
        assert call(21, ws)[2] == (capi.SPEC_ETIMEOUT if with_status else 0)
    finally:
        assert capi._lib.spec_test_stop_attend_cta(-1) == capi.SPEC_OK
    for seed in (22, 23):
        got, want = call(seed, ws), call(seed, capi.attend_workspace(D))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert got[2] == want[2] == 0


def spoiled(length, rows, Hq, Hkv, D, dtype, bs, staged, spoil, copies=None):
    """Attention of one sequence, there so often that a CTA takes whole units (or
    `copies` times), with V values put in by `spoil`: every copy against the oracle.
    bs 0: a packed prompt."""
    capi = _capi()
    n, group = rows or length, Hq // Hkv
    units = -(-n // (2 * (128 // group)))
    B = copies or 2 + 148 * 24 // (Hkv * units * (length // 128 + 4))
    k, v = (rand((length, Hkv, D), dtype, s) for s in (30, 31))
    spoil(v)
    q = rand((n, Hq, D), dtype, 32, 2.0)
    every = q.repeat(B, 1, 1).cuda()
    out, st = torch.zeros_like(every), _status()
    lse = torch.zeros((B * n, Hq), device="cuda")
    ws, off = capi.attend_workspace(D), offsets([n] * B).cuda()
    if bs == 0:
        capi.spec_attend_prompt(every, k.repeat(B, 1, 1).cuda(), v.repeat(B, 1, 1).cuda(), off, out,
                                st, ws, lse=lse)
    else:
        cached = length - n if staged else length
        pages = max(1, -(-cached // bs))
        pool = torch.full((2, pages * bs, Hkv, D), float("nan"), dtype=dtype)
        pool[0, :cached], pool[1, :cached] = k[:cached], v[:cached]
        pool = pool.view(2, pages, 1, bs, Hkv, D).permute(1, 2, 0, 3, 4, 5).contiguous().cuda()
        stage = None
        if staged:
            stage = torch.stack([k[cached:], v[cached:]], 1)[None, :, None]
            stage = stage.repeat(B, 1, 1, 1, 1, 1).cuda()
        tables = torch.arange(pages, dtype=torch.int32).repeat(B, 1).cuda()
        capi.spec_attend_paged(every, pool, 0, tables,
                               torch.full((B,), cached, dtype=torch.int32).cuda(), out, st, ws,
                               row_off=off, lse=lse, kv_stage=stage)
    torch.cuda.synchronize()
    assert int(st) == 0
    with np.errstate(invalid="ignore"):
        want = attend_rows(f64(q), f64(k), f64(v), D ** -0.5)
    fine = np.isfinite(want.out)
    odd = torch.from_numpy(np.where(fine, 0.0, want.out)).to(dtype).nan_to_num(5.0, 6.0, 7.0)
    some = ~np.isneginf(want.lse).any(1)      # rows that see a key
    w = AttendResult(np.where(fine, want.out, 0.0)[some], want.lse[some],
                     np.where(fine, want.mass, 0.0)[some], np.where(fine, want.vsum, 0.0)[some],
                     want.qk[some])
    for got, z in zip(out.view(B, n, Hq, D).cpu(), lse.view(B, n, Hq).cpu()):
        # NaN and infinities where the sum has them, and nowhere else
        at = torch.where(got.isfinite(), 0.0, got).nan_to_num(5.0, 6.0, 7.0)
        assert torch.equal(at, odd)
        check(torch.where(got.isfinite(), got, 0.0)[some], z[some], w, dtype, D)


@pytest.mark.parametrize("length,rows,Hq,Hkv,D,dtype,bs,staged,key", [
    (698, None, 1, 1, 64, torch.bfloat16, 0, False, 255),
    (443, 698, 1, 1, 128, torch.bfloat16, 16, False, 255),
    (443, 400, 4, 2, 64, torch.float16, 16, False, 383),
    (500, None, 3, 1, 96, torch.bfloat16, 0, False, 255),
    (700, None, 8, 2, 128, torch.float16, 0, False, 640),
    (300, 300, 7, 1, 64, torch.bfloat16, 24, False, 200),
    (900, 9, 32, 8, 128, torch.bfloat16, 16, True, 895),
    (137, 9, 8, 2, 64, torch.float16, 16, True, 128),
    (260, 260, 128, 1, 64, torch.bfloat16, 8, False, 130),
    (300, 200, 4, 1, 80, torch.float16, 4, False, 190),
    (210, 20, 4, 1, 128, torch.bfloat16, 3, True, 200),
    (150, 150, 2, 1, 64, torch.bfloat16, 16, True, 149),
    (131, None, 1, 1, 40, torch.bfloat16, 0, False, 0),
])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("copies", [None, 1, 6])
def test_rows_before_a_value_that_is_not_finite(length, rows, Hq, Hkv, D, dtype, bs, staged, key,
                                                value, copies):
    """A V value that is not finite reaches the rows that see it, in its column, and
    no row before it, whichever tiles and parts they share."""
    def spoil(v):
        v[key, :, 3] = value
    spoiled(length, rows, Hq, Hkv, D, dtype, bs, staged, spoil, copies)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bs,staged", [(0, False), (16, False), (16, True), (4, False)])
def test_rows_between_many_values_that_are_not_finite(dtype, bs, staged):
    """One in every column but the first two, at positions all along, also two of
    opposite sign in one column (NaN from the second on)."""
    length, rows, D = 600, (None if bs == 0 else 70), 64
    rng = np.random.default_rng(7)

    def spoil(v):
        for c in range(2, D):
            v[int(rng.integers(0, length)), int(rng.integers(0, 2)), c] = float("inf")
        for c in range(5, 20):
            v[int(rng.integers(length - 70, length)), :, c] = -float("inf")
        for c in range(40, 50):
            v[int(rng.integers(length - 70, length)), :, c] = float("nan")
    spoiled(length, rows, 8, 2, D, dtype, bs, staged, spoil)


@pytest.mark.parametrize("inplace", [False, True])
def test_extend_with_a_map_of_no_rows(inplace):
    """A slot map without elements is a map of capacity 0, not no map: rows that
    do not fit it are refused, none is what fits."""
    capi = _capi()

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")
    tables, lens, top = i32([[3, -1], [-1, -1]]), i32([5, 0]), i32([4])
    stack, st = i32([0, 1, 2, 4, 5]), _status()
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    new, ntop, off = (lens, top, i32([-9] * 3)) if inplace else (i32([-9] * 2), i32([-9]),
                                                                 i32([-9] * 3))
    before = [t.clone() for t in (tables, lens, top, new, ntop, off)]
    capi.spec_extend_paged(tables, lens, i32([0, 1]), stack, top, new, ntop, off, st,
                           slot_map=slots)
    torch.cuda.synchronize()
    assert int(st) == capi.SPEC_EINVAL
    for t, was in zip((tables, lens, top, new, ntop, off), before):
        assert torch.equal(t, was)
    st.zero_()
    capi.spec_extend_paged(tables, lens, i32([0, 0]), stack, top, new, ntop, off, st,
                           slot_map=slots)
    torch.cuda.synchronize()
    assert int(st) == 0 and new.tolist() == [5, 0] and int(ntop) == 4 and off.tolist() == [0, 0, 0]


def test_attention_over_a_staging_buffer_of_no_rows():
    """Rows beside a staging buffer that holds none are refused; without rows there
    is nothing to refuse."""
    capi = _capi()
    pool, tables = paged_inputs([40], 16, 1, 64, torch.bfloat16, 40, layers=1)
    lens, ws = torch.tensor([40], dtype=torch.int32).cuda(), capi.attend_workspace(64)
    st = _status()
    stage = torch.empty((1, 0, 1, 2, 1, 64), dtype=torch.bfloat16, device="cuda")
    for n, off in ((1, None), (2, offsets([2]).cuda())):
        q = rand((n, 2, 64), torch.bfloat16, 41).cuda()
        out = torch.full_like(q, 7.0)
        with pytest.raises(ValueError):
            capi.spec_attend_paged(q, pool, 0, tables.cuda(), lens, out, st, ws, row_off=off,
                                   kv_stage=stage)
        torch.cuda.synchronize()
        assert (out == 7).all()
    capi.spec_attend_paged(q[:0], pool, 0, tables.cuda(), lens, out[:0], st, ws,
                           row_off=offsets([0]).cuda(), kv_stage=stage)
    torch.cuda.synchronize()
    assert int(st) == 0


def test_attention_workspaces_that_are_refused():
    """A workspace whose elements do not lie one after another has less memory than
    elements; one of another type counts by its bytes."""
    capi = _capi()
    q, k = (rand((5, 2, 64), torch.bfloat16, s).cuda() for s in (50, 51))
    out, st, off = torch.full_like(q, 7.0), _status(), offsets([5]).cuda()
    n = capi.spec_attend_workspace_bytes(64)
    small, ints = torch.zeros(256, dtype=torch.uint8, device="cuda"), n // 4
    for ws in (small[:1].expand(n), torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2],
               torch.zeros((n // 256, 512), dtype=torch.uint8, device="cuda")[:, :256]):
        with pytest.raises(ValueError):
            capi.spec_attend_prompt(q, k, k, off, out, st, ws)
    with pytest.raises(capi.SpecError):
        capi.spec_attend_prompt(q, k, k, off, out, st,
                                torch.zeros(ints - 1, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert (out == 7).all() and int(st) == 0
    want = torch.empty_like(q)
    capi.spec_attend_prompt(q, k, k, off, want, st, capi.attend_workspace(64))
    capi.spec_attend_prompt(q, k, k, off, out, st,
                            torch.zeros(ints, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(out, want) and int(st) == 0


@pytest.mark.parametrize("T", [40, 200, 9000])
def test_the_cache_calls_captured_and_replayed(T):
    """Tables grown, rows stored and attended in one captured graph, replayed with
    other counts and values: one launch and two of each call, error pending or not."""
    capi = _capi()
    B, H, D, bs, cap = 3, 1, 64, 16, T
    N = B * (-(-T // bs)) + 4

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")
    tables = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
    lens, top = i32([0] * B), i32([N])
    stack, add, st = torch.randperm(N).to(torch.int32).cuda(), i32([0] * B), _status()
    off, slots = i32([0] * (B + 1)), torch.zeros(cap, dtype=torch.int64, device="cuda")
    kv = torch.zeros((cap, 2, H, D), dtype=torch.bfloat16, device="cuda")
    q = rand((cap, 2, D), torch.bfloat16, 60, 2.0).cuda()
    pool = torch.zeros((N, 1, 2, bs, H, D), dtype=torch.bfloat16, device="cuda")
    out, ws = torch.zeros_like(q), capi.attend_workspace(D)

    def calls():
        capi.spec_extend_paged(tables, lens, add, stack, top, lens, top, off, st, slot_map=slots)
        capi.spec_store_kv(kv[:, 0], kv[:, 1], slots, pool, 0, st)
        capi.spec_attend_paged(q, pool, 0, tables, lens, out, st, ws, row_off=off)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        calls()
    rows = [[torch.empty((0, H, D), dtype=torch.bfloat16)] * 2 for _ in range(B)]
    for step, n in enumerate(([T // 4, 1, T // 8], [0, T // 3, 2], [1, 1, 1])):
        new = rand((cap, 2, H, D), torch.bfloat16, 61 + step)
        kv.copy_(new)
        add.copy_(torch.tensor(n))
        graph.replay()
        torch.cuda.synchronize()
        assert int(st) == 0
        at = np.concatenate([[0], np.cumsum(n)])
        assert off.tolist() == at.tolist() and (slots[at[-1]:] == -1).all()
        for b in range(B):
            r = slice(at[b], at[b + 1])
            rows[b] = [torch.cat([x, new[r, i]]) for i, x in enumerate(rows[b])]
            assert int(lens[b]) == len(rows[b][0])
            some = slice(max(at[b], at[b + 1] - 5), at[b + 1])   # the last rows of each
            want = attend_rows(f64(q[some]), *(f64(x) for x in rows[b]), D ** -0.5)
            check(out[some], None, want, torch.bfloat16, D)
    st.fill_(capi.SPEC_ENOBLOCKS)                       # pending: the cache stays
    before = [t.clone() for t in (tables, lens, top, pool)]
    kv.fill_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    for t, was in zip((tables, lens, top, pool), before):
        assert torch.equal(t, was)
    assert int(st) == capi.SPEC_ENOBLOCKS


def test_rows_before_a_nan_beside_a_bad_table_entry():
    """The positions of a bad entry stand for rows of zeros in the columns that are
    formed again, too."""
    capi = _capi()
    n, D, bs, B = 300, 64, 16, 60
    k, v = (rand((304, 1, D), torch.bfloat16, s) for s in (70, 71))
    v[250, 0, 5:9] = float("nan")
    q = rand((n, 4, D), torch.bfloat16, 72, 2.0)
    pool = torch.stack([k, v]).view(2, 19, 1, bs, 1, D).permute(1, 2, 0, 3, 4, 5)
    tables = torch.arange(19, dtype=torch.int32)
    tables[3] = 19
    st, ws = _status(), capi.attend_workspace(D)
    every = q.repeat(B, 1, 1).cuda()
    out, lse = torch.zeros_like(every), torch.zeros((B * n, 4), device="cuda")
    capi.spec_attend_paged(every, pool.contiguous().cuda(), 0, tables.repeat(B, 1).cuda(),
                           torch.full((B,), n, dtype=torch.int32).cuda(), out, st, ws, lse=lse)
    torch.cuda.synchronize()
    assert int(st) == capi.SPEC_EDEVICE
    k[48:64], v[48:64] = 0.0, 0.0
    with np.errstate(invalid="ignore"):
        want = attend_rows(f64(q), f64(k[:n]), f64(v[:n]), D ** -0.5)
    w = AttendResult(want.out[:250], want.lse[:250], want.mass[:250], want.vsum[:250],
                     want.qk[:250])
    for got, z in zip(out.view(B, n, 4, D).cpu(), lse.view(B, n, 4).cpu()):
        check(got[:250], z[:250], w, torch.bfloat16, D)
        assert got[250:, :, 5:9].isnan().all() and got[250:, :, :5].isfinite().all()
