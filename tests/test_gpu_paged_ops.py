"""Growing block tables, storing K/V rows, and the four paged-cache operators
run together as an engine uses them, on the GPU against the oracle."""
import numpy as np
import pytest
import torch

from oracle.attend import extend_paged
from oracle.commit import check_invariants
from speculative_decoding_verification_89_b200 import workloads as W
from tests.attend_run import check_paged, check_prompt, offsets, rand

pytestmark = pytest.mark.gpu


def _capi():
    from speculative_decoding_verification_89_b200 import capi
    return capi


def _i32(v):
    return torch.as_tensor(v, dtype=torch.int32).cuda()


def run_extend(state, add, capacity, inplace=False, status=0, with_map=True):
    capi = _capi()
    B = len(add)
    t, n = state.tables.cuda(), state.seq_lens.cuda()
    f, top = state.free_stack.cuda(), state.free_top.cuda()
    new, ntop = (n, top) if inplace else (torch.full_like(n, -9), torch.full_like(top, -9))
    off = torch.full((B + 1,), -9, dtype=torch.int32, device="cuda")
    slots = torch.full((capacity,), -9, dtype=torch.int64, device="cuda") if with_map else None
    st = _i32([status])
    capi.spec_extend_paged(t, n, _i32(add), f, top, new, ntop, off, st,
                           block_size=state.block_size, slot_map=slots)
    torch.cuda.synchronize()
    return dict(tables=t.cpu(), lens=new.cpu(), top=ntop.cpu(), off=off.cpu(),
                slots=None if slots is None else slots.cpu(), status=int(st), stack=f.cpu(),
                old_lens=n.cpu(), old_top=top.cpu())


def oracle_extend(state, add, capacity):
    return extend_paged(state.tables.numpy(), state.seq_lens.numpy(), add,
                        state.free_stack.numpy(), int(state.free_top[0]), state.block_size,
                        state.free_stack.numel(), capacity)


def same_extend(got, ref, capacity):
    assert got["status"] == ref.status == 0
    assert got["lens"].tolist() == ref.lens.tolist()
    assert int(got["top"]) == ref.free_top
    assert got["off"].tolist() == ref.row_off.tolist()
    assert np.array_equal(got["tables"].numpy(), ref.tables)
    if got["slots"] is not None:
        assert np.array_equal(got["slots"].numpy(), ref.slots)


def shuffled_state(ctx, bs, max_blocks, num_blocks, seed):
    state = W.paged_state(ctx, bs, max_blocks, num_blocks)
    perm = torch.from_numpy(np.random.default_rng(seed).permutation(num_blocks).astype(np.int32))
    for t in (state.tables, state.free_stack):
        t[t >= 0] = perm[t[t >= 0].long()]
    return state


@pytest.mark.parametrize("B,bs,lo,hi,most", [
    (1, 16, 0, 0, 1), (1, 16, 511, 511, 1), (1, 1, 0, 9, 70), (3, 4, 0, 30, 20),
    (64, 16, 0, 700, 9), (5, 16, 0, 0, 3000), (300, 8, 0, 100, 30), (1500, 16, 0, 40, 40),
    (2, 24, 10, 90, 2049), (33, 128, 0, 500, 300),
])
@pytest.mark.parametrize("inplace", [False, True])
def test_extend_matches_the_oracle(B, bs, lo, hi, most, inplace):
    rng = np.random.default_rng(B * 7 + bs)
    ctx, add = rng.integers(lo, hi + 1, B), rng.integers(0, most + 1, B)
    add[0] = most
    need = int((-(-(ctx + add) // bs)).sum())
    state = shuffled_state(ctx.tolist(), bs, int((-(-(ctx + add) // bs)).max()) + 1, need + 2, B)
    cap = int(add.sum()) + int(rng.integers(0, 50))
    got = run_extend(state, add.tolist(), cap, inplace)
    same_extend(got, oracle_extend(state, add, cap), cap)
    if not inplace:    # the inputs stay
        assert torch.equal(got["old_lens"], state.seq_lens)
        assert torch.equal(got["old_top"], state.free_top)
    assert torch.equal(got["stack"], state.free_stack)
    assert check_invariants(got["tables"].numpy(), got["lens"].numpy(), state.free_stack.numpy(),
                            int(got["top"]), bs, need + 2) == []


@pytest.mark.parametrize("B,bs,most", [(3, 16, 400000), (9000, 16, 60), (4097, 1, 2),
                                       (500, 64, 2100), (4096, 16, 2), (2, 16, 4090),
                                       (2, 16, 4096)])
def test_extend_large(B, bs, most):
    """Around the limits between one launch and two."""
    rng = np.random.default_rng(B)
    ctx, add = rng.integers(0, 100, B), rng.integers(0, most + 1, B)
    need = int((-(-(ctx + add) // bs)).sum())
    state = shuffled_state(ctx.tolist(), bs, int((-(-(ctx + add) // bs)).max()), need, B)
    cap = int(add.sum()) + 5
    got = run_extend(state, add.tolist(), cap, inplace=True)
    same_extend(got, oracle_extend(state, add, cap), cap)


def test_extend_without_a_map_and_by_nothing():
    state = shuffled_state([5, 0, 16], 16, 3, 8, 1)
    got = run_extend(state, [0, 0, 0], 0)
    same_extend(got, oracle_extend(state, [0, 0, 0], 0), 0)
    got = run_extend(state, [20, 3, 1], 0, with_map=False)
    ref = oracle_extend(state, [20, 3, 1], 24)
    same_extend(got, ref, 24)


def _refusals():
    def cut(s, add, cap):      # the pool one block short
        s.free_top[0] -= 1
        return add, cap, -4
    def bad_len(s, add, cap):
        s.seq_lens[1] = -1
        return add, cap, -1
    def bad_add(s, add, cap):
        return [add[0], -1, add[2]], cap, -1
    def too_long(s, add, cap):
        return [add[0], add[1], 16 * 8], cap, -1
    def overflow(s, add, cap):
        return [2 ** 31 - 1, add[1], add[2]], cap, -1
    def no_room(s, add, cap):
        return add, cap - 1, -1
    def bad_top(s, add, cap):
        s.free_top[0] = 99
        return add, cap, -1
    def bad_entry(s, add, cap):
        s.tables[0, 0] = 40
        return add, cap, -1
    def bad_popped(s, add, cap):
        s.free_stack[int(s.free_top[0]) - 2] = -3
        return add, cap, -1
    return [cut, bad_len, bad_add, too_long, overflow, no_room, bad_top, bad_entry, bad_popped]


@pytest.mark.parametrize("spoil", _refusals(), ids=lambda f: f.__name__)
def test_extend_refusals_change_nothing(spoil):
    state = shuffled_state([5, 0, 16], 16, 8, 6, 2)     # two blocks held, four free
    add, cap, code = spoil(state, [20, 3, 17], 40)
    got = run_extend(state, add, cap)
    assert got["status"] == code
    for key, t in (("tables", state.tables), ("old_lens", state.seq_lens),
                   ("old_top", state.free_top), ("stack", state.free_stack)):
        assert torch.equal(got[key], t)
    for key in ("lens", "top", "off", "slots"):
        assert (got[key] == -9).all()


def test_extend_does_nothing_while_an_error_is_pending():
    state = shuffled_state([5, 0, 16], 16, 8, 6, 2)
    got = run_extend(state, [1, 1, 1], 3, status=-5)
    assert got["status"] == -5 and torch.equal(got["tables"], state.tables)
    assert (got["lens"] == -9).all() and (got["slots"] == -9).all()


@pytest.mark.parametrize("T,H,D,bs,layers,layer,dtype", [
    (1, 1, 8, 1, 1, 0, torch.bfloat16), (9, 8, 128, 16, 2, 1, torch.bfloat16),
    (200, 2, 64, 16, 3, 2, torch.float16), (77, 3, 40, 24, 1, 0, torch.float16),
    (1000, 1, 128, 8, 2, 0, torch.bfloat16), (5, 16, 256, 16, 2, 1, torch.bfloat16),
    (3, 9, 136, 4, 1, 0, torch.float16),
])
def test_store_moves_rows_and_nothing_else(T, H, D, bs, layers, layer, dtype):
    capi = _capi()
    N = -(-T // bs) + 3
    pool = rand((N, layers, 2, bs, H, D), dtype, 1).cuda()
    kv = rand((T, 3, H, D), dtype, 2).cuda()             # rows at a stride
    slots = torch.randperm(N * bs, generator=torch.Generator().manual_seed(3))[:T]
    slots[T // 3::5] = -1
    want = pool.clone()
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            want[s // bs, layer, 0, s % bs] = kv[t, 0]
            want[s // bs, layer, 1, s % bs] = kv[t, 2]
    st = _i32([0])
    capi.spec_store_kv(kv[:, 0], kv[:, 2], slots.cuda(), pool, layer, st)
    torch.cuda.synchronize()
    assert int(st) == 0 and torch.equal(pool, want)


def test_store_bad_slots_are_skipped_and_flagged():
    capi = _capi()
    pool = rand((4, 1, 2, 8, 2, 16), torch.bfloat16, 1).cuda()
    k = rand((4, 2, 16), torch.bfloat16, 2).cuda()
    want = pool.clone()
    want[3, 0, 0, 7], want[3, 0, 1, 7] = k[1], k[1]
    st = _i32([0])
    slots = torch.tensor([32, 31, -2, 2 ** 40], device="cuda")
    capi.spec_store_kv(k, k, slots, pool, 0, st)
    torch.cuda.synchronize()
    assert int(st) == -1 and torch.equal(pool, want)
    capi.spec_store_kv(k, k, torch.arange(4, device="cuda"), pool, 0, st)  # error pending
    torch.cuda.synchronize()
    assert torch.equal(pool, want)


def test_refusals_of_the_binding():
    capi = _capi()
    st, ws = _i32([0]), capi.attend_workspace(64)
    q = rand((4, 2, 64), torch.bfloat16, 1).cuda()
    k = rand((4, 1, 64), torch.bfloat16, 2).cuda()
    off = _i32([0, 4])
    out = torch.empty_like(q)
    for bad in (dict(q=q.float()), dict(k=k.half()), dict(off=off.long()), dict(q=q[:, :, :63]),
                dict(k=k[:3]), dict(out=out.transpose(0, 1)), dict(ws=ws.cpu())):
        a = dict(q=q, k=k, off=off, out=out, ws=ws)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            capi.spec_attend_prompt(a["q"], a["k"], k, a["off"], a["out"], st, a["ws"])
    for bad in (dict(scale=0.0), dict(scale=float("nan")), dict(scale=-1.0)):
        with pytest.raises(capi.SpecError):
            capi.spec_attend_prompt(q, k, k, off, out, st, ws, **bad)
    with pytest.raises(capi.SpecError):     # rows not on 16-byte boundaries
        wide = torch.empty((4, 2 * 64 + 4), dtype=torch.bfloat16, device="cuda")
        capi.spec_attend_prompt(wide[:, :128].unflatten(1, (2, 64)), k, k, off, out, st, ws)
    with pytest.raises(capi.SpecError):     # a workspace too small
        capi.spec_attend_prompt(q, k, k, off, out, st, ws[:1024])
    pool = rand((4, 2, 2, 16, 1, 64), torch.bfloat16, 3).cuda()
    tables, lens = _i32([[0, 1]]), _i32([20])
    with pytest.raises(ValueError):         # no such layer
        capi.spec_attend_paged(q, pool, 2, tables, lens, out, st, ws, row_off=off)
    with pytest.raises(ValueError):         # another type of cache
        capi.spec_attend_paged(q, pool.half(), 0, tables, lens, out, st, ws, row_off=off)
    with pytest.raises(ValueError):         # 4 rows do not divide over 3 sequences
        capi.spec_attend_paged(q, pool, 0, tables.repeat(3, 1), lens.repeat(3), out, st, ws)
    with pytest.raises(capi.SpecError):     # more rows than staged
        capi.spec_attend_paged(q, pool, 0, tables, lens, out, st, ws,
                               kv_stage=torch.zeros((1, 3, 2, 2, 1, 64), dtype=q.dtype,
                                                    device="cuda"))
    assert int(st) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_request_from_its_prompt_through_a_check(dtype):
    """Two requests admitted, their prompts attended and stored in the pool;
    then rounds of drafted rows attend the cache and their staged rows, and
    the commit keeps some of them. Every attention result is compared with the
    oracle's over the rows kept so far, taken from a plain list of rows."""
    capi = _capi()
    B, Hq, Hkv, D, bs, layers, layer, K = 2, 4, 2, 64, 16, 2, 1, 4
    N, max_blocks = 24, 10
    gen = np.random.default_rng(5)
    tables = torch.full((B, max_blocks), -1, dtype=torch.int32, device="cuda")
    lens, top = _i32([0] * B), _i32([N])
    stack = _i32(np.random.default_rng(6).permutation(N))
    st, ws = _i32([0]), capi.attend_workspace(D)
    pool = torch.full((N, layers, 2, bs, Hkv, D), float("nan"), dtype=dtype, device="cuda")
    prompt = [37, 64]
    T = sum(prompt)
    off = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    slots = torch.empty(T + 11, dtype=torch.int64, device="cuda")
    capi.spec_extend_paged(tables, lens, _i32(prompt), stack, top, lens, top, off, st,
                           block_size=bs, slot_map=slots)
    q, k, v = (rand((T + 11, h, D), dtype, s).cuda() for h, s in ((Hq, 1), (Hkv, 2), (Hkv, 3)))
    out = torch.zeros_like(q)
    capi.spec_attend_prompt(q, k, v, off, out, st, ws)
    capi.spec_store_kv(k, v, slots, pool, layer, st)
    torch.cuda.synchronize()
    assert int(st) == 0 and off.tolist() == [0, 37, 101] and lens.tolist() == prompt
    check_prompt(q[:T], k[:T], v[:T], prompt, out[:T], None, D ** -0.5)
    rows = [(k[:37].cpu(), v[:37].cpu()), (k[37:T].cpu(), v[37:T].cpu())]
    for step in range(4):
        stage = rand((B, K + 1, layers, 2, Hkv, D), dtype, 10 + step).cuda()
        q = rand((B * (K + 1), Hq, D), dtype, 20 + step, 2.0).cuda()
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
        capi.spec_attend_paged(q, pool, layer, tables, lens, out, st, ws, kv_stage=stage, lse=lse)
        # what the oracle sees: the rows kept so far, as a pool of one block each
        for b in range(B):
            kk, vv = rows[b]
            one = torch.stack([kk, vv])[None, None]
            check_paged(q[b * (K + 1):(b + 1) * (K + 1)], one, 0,
                        torch.zeros((1, 1), dtype=torch.int32), [len(kk)], [K + 1],
                        out[b * (K + 1):(b + 1) * (K + 1)], lse[b * (K + 1):(b + 1) * (K + 1)],
                        D ** -0.5, stage[b:b + 1, :, layer:layer + 1])
        keep = _i32(gen.integers(0, K + 1, B))
        capi.spec_commit_paged(tables, lens, None, keep, 1, stack, top, K + 1, st, block_size=bs,
                               kv_stage=stage, kv_pool=pool)
        torch.cuda.synchronize()
        assert int(st) == 0
        for b in range(B):
            n = int(keep[b]) + 1
            rows[b] = tuple(torch.cat([x, stage[b, :n, layer, i].cpu()])
                            for i, x in enumerate(rows[b]))
        assert lens.tolist() == [len(r[0]) for r in rows]
        assert check_invariants(tables.cpu().numpy(), lens.cpu().numpy(), stack.cpu().numpy(),
                                int(top), bs, N) == []
