"""Prompt and paged attention on the GPU against the fp64 oracle, through the
C ABI: head layouts, lengths, strides, ragged batches, empty rows, what lies
in masked places, streams and graphs."""
import numpy as np
import pytest
import torch

from tests.attend_run import (check_paged, check_prompt, deal_tables, offsets, rand)

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def _capi():
    from speculative_decoding_verification_89_b200 import capi
    return capi


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def run_prompt(q, k, v, lens, scale=None, want_lse=True, off=None, ws=None, **kw):
    capi = _capi()
    T, Hq, D = q.shape
    out = torch.full((T, Hq, D), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda") if want_lse else None
    st = _status()
    ws = capi.attend_workspace(D) if ws is None else ws
    capi.spec_attend_prompt(q, k, v, (offsets(lens) if off is None else off).cuda(), out, st, ws,
                            scale=scale, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse, int(st)


def run_paged(q, pool, layer, tables, lens, rows=None, stage=None, scale=None):
    capi = _capi()
    T, Hq, D = q.shape
    out = torch.full((T, Hq, D), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    st = _status()
    capi.spec_attend_paged(q, pool, layer, tables.cuda(),
                           torch.tensor(lens, dtype=torch.int32).cuda(), out, st,
                           capi.attend_workspace(D), kv_stage=stage, scale=scale, lse=lse,
                           row_off=None if rows is None else offsets(rows).cuda())
    torch.cuda.synchronize()
    return out, lse, int(st)


def prompt_inputs(lens, Hq, Hkv, D, dtype, seed, extra=0):
    T = sum(lens) + extra
    return (rand((T, Hq, D), dtype, seed, 2.0).cuda(), rand((T, Hkv, D), dtype, seed + 1).cuda(),
            rand((T, Hkv, D), dtype, seed + 2).cuda())


PROMPTS = [
    ([1], 1, 1, 128, BF), ([128], 1, 1, 128, BF), ([129], 4, 1, 64, FP),
    ([5, 1, 0, 33], 4, 2, 128, BF), ([97], 8, 1, 64, FP), ([64, 257], 8, 2, 128, FP),
    ([300, 1, 127], 3, 1, 96, BF), ([130, 41], 7, 1, 80, FP), ([40, 19], 5, 5, 8, BF),
    ([500], 16, 1, 128, BF), ([33], 128, 1, 64, BF), ([31, 200], 48, 1, 72, FP),
    ([700], 2, 2, 128, BF),
]


@pytest.mark.parametrize("lens,Hq,Hkv,D,dtype", PROMPTS)
def test_prompt(lens, Hq, Hkv, D, dtype):
    q, k, v = prompt_inputs(lens, Hq, Hkv, D, dtype, 100 + sum(lens) + D)
    out, lse, st = run_prompt(q, k, v, lens)
    assert st == 0
    check_prompt(q, k, v, lens, out, lse, D ** -0.5)


@pytest.mark.parametrize("trial", range(6))
def test_prompt_random(trial):
    rng = np.random.default_rng(trial)
    lens = rng.integers(0, 260, size=int(rng.integers(1, 7))).tolist() + [1]
    Hkv = int(rng.integers(1, 4))
    Hq = Hkv * int(rng.integers(1, 10))
    D = 8 * int(rng.integers(1, 17))
    q, k, v = prompt_inputs(lens, Hq, Hkv, D, (BF, FP)[trial % 2], trial)
    out, lse, st = run_prompt(q, k, v, lens, scale=0.7 * D ** -0.5)
    assert st == 0
    check_prompt(q, k, v, lens, out, lse, 0.7 * D ** -0.5)


def test_prompt_peaked_and_large_scores():
    """Scores of some hundreds, growing along the keys, so the reference is
    raised again and again, and one row far above the others."""
    lens = [600]
    q, k, v = prompt_inputs(lens, 4, 2, 128, BF, 5)
    k = k * torch.linspace(0.1, 6.0, 600, device="cuda").to(BF)[:, None, None]
    k[77] *= 8
    out, lse, st = run_prompt(q, k, v, lens)
    assert st == 0
    check_prompt(q, k, v, lens, out, lse, 128 ** -0.5)


def test_prompt_strided_rows_of_one_projection():
    lens, Hq, Hkv, D = [70, 150], 8, 2, 64
    T = sum(lens)
    qkv = rand((T, (Hq + 2 * Hkv) * D + 8), BF, 3).cuda()
    q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    k = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    v = qkv[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].unflatten(1, (Hkv, D))
    out, lse, st = run_prompt(q, k, v, lens)
    assert st == 0
    check_prompt(q, k, v, lens, out, lse, D ** -0.5)


def test_prompt_rows_behind_the_last_sequence_stay():
    """Rows outside every sequence are neither read (they hold NaN) nor written,
    nor do a neighbour's NaN rows reach a sequence."""
    lens = [40, 130]
    q, k, v = prompt_inputs(lens, 4, 1, 128, BF, 8, extra=9)
    for t in (q, k, v):
        t[170:] = float("nan")
        t[:40] = float("nan")
    out, lse, st = run_prompt(q, k, v, lens)
    assert st == 0
    assert (out[170:] == 7).all() and (lse[170:] == 7).all()
    assert out[:40].isnan().all()
    check_prompt(q[40:170], k[40:170], v[40:170], [130], out[40:170], lse[40:170], 128 ** -0.5)


def test_prompt_invalid_ranges_are_left_out():
    """A range that decreases and one past T are left out and flagged; the
    valid ones between are attended."""
    q, k, v = prompt_inputs([80], 2, 1, 64, BF, 9)
    off = torch.tensor([0, 30, 20, 75, 81], dtype=torch.int32)
    out, lse, st = run_prompt(q, k, v, None, off=off)
    assert st == -6
    assert (out[75:] == 7).all()
    check_prompt(q[:20], k[:20], v[:20], [20], out[:20], lse[:20], 64 ** -0.5)


def test_prompt_same_bits_every_time_and_without_lse():
    lens = [1000, 37]
    q, k, v = prompt_inputs(lens, 8, 2, 128, BF, 10)
    a, la, _ = run_prompt(q, k, v, lens)
    b, lb, _ = run_prompt(q, k, v, lens)
    c, _, _ = run_prompt(q, k, v, lens, want_lse=False)
    assert torch.equal(a, b) and torch.equal(la, lb) and torch.equal(a, c)


def test_prompt_many_short_sequences():
    """More sequences than threads of a block, many of them empty."""
    rng = np.random.default_rng(11)
    lens = rng.integers(0, 4, 900).tolist()
    q, k, v = prompt_inputs(lens, 4, 2, 64, FP, 12)
    out, lse, st = run_prompt(q, k, v, lens)
    assert st == 0
    check_prompt(q, k, v, lens, out, lse, 64 ** -0.5)


def test_no_rows_at_all():
    q, k, v = prompt_inputs([0, 0], 2, 1, 64, BF, 13, extra=5)
    out, lse, st = run_prompt(q, k, v, [0, 0])
    assert st == 0 and (out == 7).all() and (lse == 7).all()


def test_one_workspace_for_several_head_sizes():
    """Calls of other sizes in turn on one workspace, units divided over CTAs in
    each, give what a workspace of their own gives."""
    ws = _capi().attend_workspace(128)
    for rnd in range(2):
        for lens, D in (([700, 30], 128), ([900], 64), ([256, 700], 96)):
            q, k, v = prompt_inputs(lens, 4, 1, D, BF, 14 + D)
            a, la, _ = run_prompt(q, k, v, lens, ws=ws)
            b, lb, st = run_prompt(q, k, v, lens)
            assert st == 0 and torch.equal(a, b) and torch.equal(la, lb)


def paged_inputs(lens, bs, Hkv, D, dtype, seed, layers=2, extra=3):
    nb = sum(-(-n // bs) for n in lens) + extra
    max_blocks = max([-(-n // bs) for n in lens] + [1]) + 1
    pool = rand((nb, layers, 2, bs, Hkv, D), dtype, seed).cuda()
    return pool, deal_tables(lens, bs, nb, max_blocks, seed)


PAGED = [
    # lens, rows (None: one each), block size, Hq, Hkv, D, dtype
    ([1], None, 16, 1, 1, 128, BF), ([700], None, 16, 8, 2, 128, BF),
    ([1, 17, 300], None, 16, 4, 1, 64, FP), ([513, 2, 128], [3, 1, 9], 16, 8, 2, 128, BF),
    ([400, 90], [200, 90], 16, 4, 2, 128, FP), ([260], [260], 8, 4, 4, 64, BF),
    ([33, 5, 77], [0, 5, 1], 1, 3, 1, 40, BF), ([250, 129], [7, 129], 24, 6, 2, 128, BF),
    ([300], [40], 64, 7, 1, 96, FP), ([1000], [1], 128, 16, 1, 128, BF),
    ([900, 11], None, 256, 32, 1, 128, BF), ([130], [2], 3, 128, 1, 64, FP),
    ([500, 384], [1, 50], 384, 4, 2, 120, FP), ([290], [3], 100, 4, 1, 88, BF),
]


@pytest.mark.parametrize("lens,rows,bs,Hq,Hkv,D,dtype", PAGED)
def test_paged(lens, rows, bs, Hq, Hkv, D, dtype):
    pool, tables = paged_inputs(lens, bs, Hkv, D, dtype, 50 + sum(lens))
    n = rows or [1] * len(lens)
    q = rand((sum(n), Hq, D), dtype, 60 + sum(lens), 2.0).cuda()
    out, lse, st = run_paged(q, pool, 1, tables, lens, rows)
    assert st == 0
    check_paged(q, pool, 1, tables, lens, n, out, lse, D ** -0.5)


STAGED = [
    ([700, 1, 0, 130], 9, 16, 8, 2, 128, BF), ([0], 1, 16, 4, 1, 64, FP),
    ([127, 128, 129], 5, 16, 4, 4, 128, BF), ([300], 200, 16, 4, 1, 128, FP),
    ([50, 260], 3, 5, 6, 2, 80, BF),
]


@pytest.mark.parametrize("lens,n,bs,Hq,Hkv,D,dtype", STAGED)
@pytest.mark.parametrize("ragged", [False, True])
def test_paged_staged(lens, n, bs, Hq, Hkv, D, dtype, ragged):
    pool, tables = paged_inputs(lens, bs, Hkv, D, dtype, 70 + sum(lens))
    rows = [max(0, n - 2 * b) for b in range(len(lens))] if ragged else [n] * len(lens)
    stage = rand((len(lens), n, 2, 2, Hkv, D), dtype, 71).cuda()
    q = rand((sum(rows), Hq, D), dtype, 72, 2.0).cuda()
    out, lse, st = run_paged(q, pool, 0, tables, lens, rows if ragged else None, stage)
    assert st == 0
    check_paged(q, pool, 0, tables, lens, rows, out, lse, D ** -0.5, stage)


def test_paged_long_cache_split_over_the_gpu():
    lens = [20000, 3, 6001]
    pool, tables = paged_inputs(lens, 16, 2, 128, BF, 80, layers=1)
    q = rand((3, 8, 128), BF, 81, 2.0).cuda()
    out, lse, st = run_paged(q, pool, 0, tables, lens)
    assert st == 0
    check_paged(q, pool, 0, tables, lens, [1, 1, 1], out, lse, 128 ** -0.5)


def test_paged_rows_that_see_nothing():
    """More rows than cached positions: the first rows see nothing (0, -inf);
    an empty cache leaves all of them empty."""
    lens, rows = [3, 0, 200], [5, 4, 200]
    pool, tables = paged_inputs(lens, 16, 2, 64, BF, 82)
    q = rand((sum(rows), 4, 64), BF, 83).cuda()
    out, lse, st = run_paged(q, pool, 1, tables, lens, rows)
    assert st == 0
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all()
    assert (out[5:9] == 0).all() and torch.isneginf(lse[5:9]).all()
    check_paged(q, pool, 1, tables, lens, rows, out, lse, 64 ** -0.5)


def test_paged_what_lies_past_the_end_is_not_seen():
    """Slots behind the last position and blocks no sequence holds are NaN
    (K and V); entries behind a table's end are out of range."""
    lens = [37, 130, 16]
    pool, tables = paged_inputs(lens, 16, 2, 128, BF, 84)
    held = torch.zeros(pool.shape[0], 16, dtype=torch.bool)
    for b, n in enumerate(lens):
        for p in range(n):
            held[tables[b, p // 16], p % 16] = True
    pool.masked_fill_(~held.cuda()[:, None, None, :, None, None], float("nan"))
    q = rand((3, 8, 128), BF, 85).cuda()
    out, lse, st = run_paged(q, pool, 0, tables, lens)
    assert st == 0
    check_paged(q, pool, 0, tables, lens, [1, 1, 1], out, lse, 128 ** -0.5)


@pytest.mark.parametrize("bs", [4, 8, 12, 24, 32, 40, 96, 128, 136, 200, 384])
@pytest.mark.parametrize("staged", [False, True])
def test_paged_block_sizes(bs, staged):
    """Pages that a tile divides into copies of 8 rows up to 128 and pages left
    to the row copies, ending and beginning inside a tile; more than 32 pages, a
    sequence of whole pages; what no sequence holds is NaN."""
    lens, rows = [bs * 40 + 5, 1, 10 * bs, 129], [1, 1, 4, 7]
    pool, tables = paged_inputs(lens, bs, 2, 128, BF, 300 + bs)
    held = torch.zeros(pool.shape[0], bs, dtype=torch.bool)
    for b, n in enumerate(lens):
        for p in range(n):
            held[tables[b, p // bs], p % bs] = True
    pool.masked_fill_(~held.cuda()[:, None, None, :, None, None], float("nan"))
    stage = rand((4, 7, 2, 2, 2, 128), BF, 301).cuda() if staged else None
    q = rand((sum(rows), 8, 128), BF, 302, 2.0).cuda()
    out, lse, st = run_paged(q, pool, 1, tables, lens, rows, stage)
    assert st == 0
    check_paged(q, pool, 1, tables, lens, rows, out, lse, 128 ** -0.5, stage)


def test_paged_invalid_values_are_flagged():
    """A bad length sees nothing; a bad table entry stands for zeros."""
    lens = [64, 200, -1, 40]
    pool, tables = paged_inputs([64, 96, 0, 40], 16, 1, 64, BF, 86)
    q = rand((4, 2, 64), BF, 87).cuda()
    out, lse, st = run_paged(q, pool, 0, tables, lens)   # 200 > 7 blocks of 16
    assert st == -6
    for b in (1, 2):
        assert (out[b] == 0).all() and torch.isneginf(lse[b]).all()
    check_paged(q[:1], pool, 0, tables[:1], [64], [1], out[:1], lse[:1], 64 ** -0.5)
    tables[3, 1] = pool.shape[0]
    out, lse, st = run_paged(q[3:], pool, 0, tables[3:], [40])
    assert st == -6
    zeroed = torch.cat([pool, torch.zeros_like(pool[:1])])
    check_paged(q[3:], zeroed, 0, tables[3:], [40], [1], out, lse, 64 ** -0.5)


def test_attention_captured_and_replayed_on_another_stream():
    capi = _capi()
    lens, rows = [400, 77], [3, 9]
    pool, tables = paged_inputs(lens, 16, 2, 128, BF, 88)
    q = rand((12, 8, 128), BF, 89).cuda()
    out, lse, _ = run_paged(q, pool, 1, tables, lens, rows)
    t, n, off = tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), offsets(rows).cuda()
    o2, l2, st = torch.zeros_like(out), torch.zeros_like(lse), _status()
    ws = capi.attend_workspace(128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        capi.spec_attend_paged(q, pool, 1, t, n, o2, st, ws, row_off=off, lse=l2)
    for _ in range(2):
        o2.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, out) and torch.equal(l2, lse) and int(st) == 0
    # other lengths in the same buffers: the graph works them out on the device
    n.copy_(torch.tensor([333, 20], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    check_paged(q, pool, 1, tables, [333, 20], rows, o2, l2, 128 ** -0.5)


def test_two_calls_at_once_with_a_workspace_each():
    capi = _capi()
    lens = [900, 300]
    q, k, v = prompt_inputs(lens, 8, 2, 128, BF, 90)
    want, _, _ = run_prompt(q, k, v, lens)
    off = offsets(lens).cuda()
    outs = [torch.zeros_like(want) for _ in range(4)]
    ws = [capi.attend_workspace(128) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    st = _status()
    torch.cuda.synchronize()
    for i in range(4):
        capi.spec_attend_prompt(q, k, v, off, outs[i], st, ws[i % 2], stream=streams[i % 2])
    torch.cuda.synchronize()
    assert int(st) == 0 and all(torch.equal(o, want) for o in outs)


def test_fp16_weights_far_below_the_largest():
    """One key's score is 16.25 above all others (scores exact in fp16 products),
    so theirs are weights of w = e^-16.25 = 1.47 * 2^-24 of the largest: half a
    subnormal step, were the largest 1. Weights are kept at up to 2^7 of a new
    reference, so each is off by at most 2^-25 / 2^7; outputs once more by 2^-11
    relative, sums and exponentials by less than 2^-18."""
    n, D = 256, 64
    q, k, v = (torch.zeros(n, 1, D, dtype=FP, device="cuda") for _ in range(3))
    q[:, 0, 0], k[0, 0, 0] = 4.0, 4.0625
    v[1:] = 1024.0
    out, lse, st = run_prompt(q, k, v, [n], scale=1.0)
    w, i = np.exp(-16.25), np.arange(n)
    want = 1024.0 * i * w / (1 + i * w)
    got = out.double().cpu().numpy()[:, 0]
    tol = want * (2.0 ** -32 / w + 2.0 ** -11 + 2.0 ** -18) + 2.0 ** -25
    assert st == 0 and (np.abs(got - want[:, None]) <= tol[:, None]).all()
    np.testing.assert_allclose(lse.cpu().numpy()[:, 0], 16.25 + np.log1p(i * w), rtol=2.0 ** -20)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 70])
@pytest.mark.parametrize("D", [64, 96, 128])
def test_paged_divided_units_of_any_number_of_rows(rows, D):
    """One sequence under one head, so every tile of keys goes to another CTA and
    each unit is joined from as many parts: 4 query heads of 1 to 70 rows, up to
    three units, the last of few rows."""
    pool, tables = paged_inputs([2500], 16, 1, D, BF, 400 + rows)
    q = rand((rows, 4, D), BF, 401, 2.0).cuda()
    out, lse, st = run_paged(q, pool, 0, tables, [2500], [rows])
    assert st == 0
    check_paged(q, pool, 0, tables, [2500], [rows], out, lse, D ** -0.5)


@pytest.mark.parametrize("trial", range(8))
@pytest.mark.parametrize("staged", [False, True])
def test_paged_random(trial, staged):
    """Units of one and of two tiles, without keys and with many, in one call:
    more rows than positions, single rows, chunks; the same bits on a second run."""
    rng = np.random.default_rng(500 + trial)
    B = int(rng.integers(3, 30))
    lens = rng.choice([0, 1, 5, 127, 128, 129, 700, 1500], B).tolist()
    rows = rng.choice([0, 1, 2, 9, 33, 64, 65, 150], B).tolist() + [1]
    lens.append(300)
    Hkv, G, D = int(rng.integers(1, 4)), int(rng.choice([1, 2, 4, 7])), int(rng.choice([64, 80, 128]))
    dtype = (BF, FP)[trial % 2]
    pool, tables = paged_inputs(lens, int(rng.choice([8, 16, 24, 64])), Hkv, D, dtype, 600 + trial)
    stage = rand((B + 1, 150, 2, 2, Hkv, D), dtype, 601).cuda() if staged else None
    q = rand((sum(rows), Hkv * G, D), dtype, 602, 2.0).cuda()
    out, lse, st = run_paged(q, pool, 1, tables, lens, rows, stage)
    again, lse2, _ = run_paged(q, pool, 1, tables, lens, rows, stage)
    assert st == 0 and torch.equal(out, again) and torch.equal(lse, lse2)
    check_paged(q, pool, 1, tables, lens, rows, out, lse, D ** -0.5, stage)


def test_two_streams_at_once_and_two_graphs_on_one_workspace():
    """Calls in flight together on workspaces of their own, and two captured
    graphs that share one replayed in turn, give what each gives alone."""
    capi = _capi()
    big, small = [3000, 17], [40, 900, 3]
    a, b = prompt_inputs(big, 8, 2, 128, BF, 700), prompt_inputs(small, 4, 1, 64, FP, 710)
    want = [run_prompt(*x, n)[0] for x, n in ((a, big), (b, small))]
    off = [offsets(n).cuda() for n in (big, small)]
    out = [torch.empty_like(x[0]) for x in (a, b)]
    ws = [capi.attend_workspace(128), capi.attend_workspace(64)]
    st, streams = _status(), [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                capi.spec_attend_prompt(*x, off[i], out[i], st, ws[i])
    torch.cuda.synchronize()
    assert int(st) == 0 and all(torch.equal(o, w) for o, w in zip(out, want))
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for i, x in enumerate((a, b)):
        with torch.cuda.graph(graphs[i], stream=streams[0]):
            capi.spec_attend_prompt(*x, off[i], out[i], st, ws[0])
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert int(st) == 0 and all(torch.equal(o, w) for o, w in zip(out, want))
