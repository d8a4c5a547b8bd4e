"""Pins of the attention / table-growth oracle: closed forms on the CPU."""
import numpy as np
import pytest

from oracle.attend import attend_rows, cached_rows, extend_paged


def test_equal_scores_average_the_keys_seen():
    n, L, D = 3, 5, 4
    v = np.arange(L * D, dtype=float).reshape(L, 1, D)
    r = attend_rows(np.zeros((n, 2, D)), np.ones((L, 1, D)), v, 0.5)
    for i in range(n):
        seen = L - n + i + 1
        assert np.allclose(r.out[i, 0], v[:seen, 0].mean(0), rtol=1e-14)
        assert np.allclose(r.lse[i], np.log(seen), rtol=1e-14)


def test_one_key_and_no_key():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(2, 4, 8)), rng.normal(size=(1, 2, 8)), rng.normal(size=(1, 2, 8))
    r = attend_rows(q, k, v, 0.3)          # two rows, one key: the first sees nothing
    assert (r.out[0] == 0).all() and (r.lse[0] == -np.inf).all()
    for h in range(4):
        assert np.allclose(r.out[1, h], v[0, h // 2])
        assert np.isclose(r.lse[1, h], 0.3 * (q[1, h] @ k[0, h // 2]))


def test_parts_join_by_their_log_sum_exp():
    """Attention over all keys equals the parts' mean weighted by exp(lse)."""
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(1, 1, 8)), rng.normal(size=(9, 1, 8)), rng.normal(size=(9, 1, 8))
    whole = attend_rows(q, k, v, 1.0)
    a, b = attend_rows(q, k[:4], v[:4], 1.0), attend_rows(q, k[4:], v[4:], 1.0)
    w = np.exp(a.lse - np.logaddexp(a.lse, b.lse))[..., None]
    assert np.allclose(whole.out, w * a.out + (1 - w) * b.out)
    assert np.allclose(whole.lse, np.logaddexp(a.lse, b.lse))


def test_cached_rows_follow_the_table():
    pool = np.arange(4 * 2 * 2 * 1 * 1, dtype=float).reshape(4, 2, 2, 1, 1)
    k, v = cached_rows(pool, [3, 0], 3)
    assert k.ravel().tolist() == [pool[3, 0, 0, 0, 0], pool[3, 0, 1, 0, 0], pool[0, 0, 0, 0, 0]]
    assert v.ravel().tolist() == [pool[3, 1, 0, 0, 0], pool[3, 1, 1, 0, 0], pool[0, 1, 0, 0, 0]]


def test_extend_worked_example():
    # blocks of 4; sequence 0 holds 5 rows in blocks 7, 2; sequence 1 nothing
    tables = np.array([[7, 2, -1], [-1, -1, -1]])
    r = extend_paged(tables, [5, 0], [4, 2], np.array([9, 1, 4, 0, 0, 0, 0, 0, 0, 0]), 3, 4, 10, 8)
    assert r.status == 0 and r.lens.tolist() == [9, 2] and r.free_top == 1
    assert r.tables.tolist() == [[7, 2, 4], [1, -1, -1]]
    assert r.row_off.tolist() == [0, 4, 6]
    assert r.slots.tolist() == [9, 10, 11, 16, 4, 5, -1, -1]


@pytest.mark.parametrize("kw,code", [
    (dict(add_len=[-1, 0]), -1), (dict(seq_lens=[-1, 0]), -1), (dict(add_len=[8, 0]), -1),
    (dict(add_len=[4, 5]), -1), (dict(free_top=0), -4), (dict(free_top=11), -1),
    (dict(tables=np.array([[7, 12, -1], [-1, -1, -1]])), -1),
])
def test_extend_refusals(kw, code):
    a = dict(tables=np.array([[7, 2, -1], [-1, -1, -1]]), seq_lens=[5, 0], add_len=[4, 2],
             free_stack=np.array([9, 1, 4, 0, 0, 0, 0, 0, 0, 0]), free_top=3, block_size=4,
             num_blocks=10, capacity=8)
    a.update(kw)
    r = extend_paged(**a)
    assert r.status == code and r.tables.tolist() == np.asarray(a["tables"]).tolist()
