"""Errors of the paged-cache and attention calls on the GPU: what a bad value
leaves done and undone, and what the next call finds."""
import pytest
import torch

from tests.attend_run import offsets, rand
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
