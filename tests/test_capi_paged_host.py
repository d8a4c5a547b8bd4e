"""Host-side refusals of the paged-cache and attention entry points: bad
arguments return before any launch (the pointers are fake and never read)."""
import ctypes

import pytest

from speculative_decoding_verification_89_b200 import build as build_mod

P, I, I64, SZ, F = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t,
                    ctypes.c_float)
fake, odd = P(0x10000), P(0x10008)


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(build_mod.build())


def refuses(f, base, cases):
    for i, v, code in cases:
        bad = list(base)
        bad[i] = v
        assert f(*bad) == code, (i, v)


def test_extend(lib):
    f = lib.spec_extend_paged
    f.restype, f.argtypes = I, [I, I, I, P, P, P, P, P, I, P, P, P, P, I64, P, P]
    base = [4, 16, 8, fake, fake, fake, fake, fake, 64, fake, fake, fake, fake, 100, fake, None]
    assert f(0, *base[1:]) == 0
    refuses(f, base, [(0, -1, -1), (0, 16385, -1), (1, 0, -1), (2, 0, -1), (2, 1 << 27, -1),
                      (8, 0, -1), (13, -1, -1), (12, P(0x10004), -1)] +
            [(i, None, -1) for i in (3, 4, 5, 6, 7, 9, 10, 11, 14)])


def test_store(lib):
    f = lib.spec_store_kv
    f.restype = I
    f.argtypes = [P, I64, P, I64, I, P, P, I, I, I, I, I, I, P, P]
    base = [fake, 1024, fake, 1024, 5, fake, fake, 64, 2, 1, 16, 8, 128, None, None]
    assert f(*base[:4], 0, *base[5:]) == 0
    refuses(f, base, [(0, None, -1), (0, odd, -1), (1, 1023, -1), (1, 1028, -1), (2, odd, -1),
                      (3, 512, -1), (4, -1, -1), (5, None, -1), (5, P(0x10004), -1),
                      (6, None, -1), (6, odd, -1), (7, 0, -1), (8, 0, -1), (9, 2, -1),
                      (9, -1, -1), (10, 0, -1), (11, 0, -1), (12, 0, -1)])
    bad = list(base)
    bad[11], bad[12] = 1, 4          # rows of 8 bytes
    assert f(*bad) == -1


def test_attend_workspace(lib):
    g = lib.spec_attend_workspace_bytes
    g.restype, g.argtypes = SZ, [I]
    assert g(128) > g(64) > 0 and g(64) % 256 == 0 and g(8) == g(64) and g(72) == g(128)
    assert g(0) == g(129) == g(136) == g(12) == 0


def test_attend_prompt(lib):
    f = lib.spec_attend_prompt
    f.restype = I
    f.argtypes = [P, I64, P, I64, P, I64, I, P, I, I, I, I, I, F, P, I64, P, P, P, SZ, P]
    base = [fake, 1024, fake, 256, fake, 256, 1, fake, 3, 100, 8, 2, 128, 0.1, fake, 1024, None,
            None, fake, 1 << 30, None]
    assert f(*base[:8], 0, *base[9:]) == 0 and f(*base[:9], 0, *base[10:]) == 0
    refuses(f, base, [(0, None, -1), (0, odd, -1), (1, 1016, -1), (1, 1028, -1), (2, None, -1),
                      (3, 255, -1), (4, odd, -1), (5, 260, -1), (6, 0, -1), (6, 3, -1),
                      (7, None, -1), (8, -1, -1), (8, 16385, -1), (9, -1, -1),
                      (9, (1 << 30) + 1, -1), (10, 7, -1), (10, 0, -1), (11, 0, -1), (11, 16, -1),
                      (12, 132, -1), (12, 12, -1), (12, 0, -1), (13, 0.0, -1), (13, -1.0, -1),
                      (13, float("inf"), -1), (13, float("nan"), -1), (13, 3e38, -1), (14, None, -1),
                      (14, odd, -1), (15, 1000, -1), (18, None, -3), (18, P(0x10010), -3),
                      (19, 1000, -3)])


def test_attend_paged(lib):
    f = lib.spec_attend_paged
    f.restype = I
    f.argtypes = [P, I64, I, P, I, I, I, I, P, I, I, I, I, I, I, P, I, P, P, I, F, P, I64, P, P,
                  P, SZ, P]
    base = [fake, 1024, 2, None, 3, 4, 12, 8, fake, 64, 2, 1, 16, 2, 128, fake, 9, fake, fake, 3,
            0.1, fake, 1024, None, None, fake, 1 << 30, None]
    bad = list(base)
    bad[5] = bad[6] = 0
    assert f(*bad) == 0                                     # B = 0
    refuses(f, base, [(0, None, -1), (1, 1000, -1), (2, 0, -1), (4, 2, -1), (4, 4, -1),
                      (4, -1, -1), (5, -1, -1), (6, 13, -1), (7, 9, -1), (7, 258, -1),
                      (8, None, -1), (8, odd, -1), (9, 0, -1), (10, 0, -1), (11, 2, -1),
                      (11, -1, -1), (12, 0, -1), (13, 0, -1), (14, 100, -1), (15, None, -1),
                      (16, 0, -1), (16, 1 << 28, -1), (17, None, -1), (18, odd, -1), (19, 2, -1),
                      (19, 0, -1), (20, 0.0, -1), (21, odd, -1), (22, 8, -1), (25, None, -3),
                      (26, 0, -3)])


def test_logit_entries_refuse_the_attention_type(lib):
    g = lib.spec_workspace_bytes
    g.restype = SZ
    assert g(4, 3, 1000, 2, 0) == 0
    h = lib.spec_draft_workspace_bytes
    h.restype = SZ
    assert h(4, 1000, 2) == 0
