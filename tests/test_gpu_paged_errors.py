"""Errors of the paged-cache and attention calls on the GPU: what a bad value
leaves done and undone, and what the next call finds."""
import pytest
import torch

from tests.attend_run import rand

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
