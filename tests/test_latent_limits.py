"""Sizes of the latent attention entry points at their limits, without a GPU: what no grid can hold is refused before
anything is launched, and nothing to do is no error."""
import ctypes

import pytest

f = ctypes.c_void_p(0x100000)  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def C():
    import compressed_sparse_kv_csa_b200 as C
    return C


def kv(C, n=64, c=576, rd=64):
    return ctypes.byref(C._KvRows(0x100000, 0x200000, 0x300000, n, c, rd))


def test_rows_that_no_grid_holds(C):
    def append(n):
        return C.lib().latent_append(f, 1, n, None, 0.0, 0.0, f, f, 4, f, 2, 16, None, kv(C), None)

    def gather(n):
        return C.lib().latent_gather(kv(C), f, None, 2, f, 2, 16, None, n, f, f, 1, None)
    for n in ((1 << 38) + 1, 1 << 40, (1 << 62) + 7):
        assert append(n) == C.CSA_ERR_UNSUPPORTED
    for n in (32 * (2 ** 31 - 1) + 1, (1 << 36) - 31, 1 << 36, 1 << 62):
        assert gather(n) == C.CSA_ERR_UNSUPPORTED


def test_nothing_to_do(C):
    """Empty arrays have no address: a call of no rows, sequences or queries needs none, and every other check still counts."""
    ok, bad = C.CSA_OK, C.CSA_ERR_INVALID_ARG
    a = C.lib().latent_append
    assert a(None, 1, 0, f, 1e-6, 1e4, None, None, 0, None, 0, 0, None, kv(C), None) == ok
    assert a(None, 1, 0, f, 1e-6, 1e4, None, None, 0, None, 0, 0, None, None, None) == bad
    assert a(None, 1, 0, f, -1.0, 1e4, None, None, 0, None, 0, 0, None, kv(C), None) == bad
    assert a(None, 1, 1, f, 1e-6, 1e4, f, None, 1, f, 2, 16, None, kv(C), None) == bad
    assert a(f, 1, 1, f, 1e-6, 1e4, None, None, 1, f, 2, 16, None, kv(C), None) == bad
    assert a(f, 1, 1, f, 1e-6, 1e4, f, None, 1, None, 2, 16, None, kv(C), None) == bad
    g = C.lib().latent_gather
    assert g(kv(C), f, None, 0, None, 0, 0, None, 0, None, None, 1, None) == ok
    assert g(kv(C), f, None, 2, f, 2, 16, None, 0, None, None, 1, None) == ok
    assert g(kv(C), f, None, 0, None, 0, 0, None, 4, f, None, 1, None) == ok
    assert g(kv(C), f, None, 0, None, 0, 0, None, 4, None, None, 1, None) == bad
    assert g(kv(C), None, None, 0, None, 0, 0, None, 0, None, None, 1, None) == bad
    assert g(kv(C), f, None, 2, None, 2, 16, None, 4, f, f, 1, None) == bad
    d = C.lib().latent_attn_decode
    assert d(None, kv(C), None, None, 0, 0, None, 1.0, 0, 1, 16, 64, None, None, None, 0, None) == ok
    assert d(None, kv(C), None, None, 0, 0, None, 1.0, 0, 1, 0, 64, None, None, None, 0, None) == bad
    assert d(None, kv(C), f, f, 2, 16, None, 1.0, 1, 1, 16, 64, f, None, f, 1 << 30, None) == bad
    assert d(f, kv(C), f, None, 2, 16, None, 1.0, 1, 1, 16, 64, f, None, f, 1 << 30, None) == bad
    p = C.lib().latent_attn_prefill
    assert p(None, f, f, f, f, 1, 0, 9, 4, 128, 64, 128, 0, 1.0, 1, 1, None, None, None, 0, None) == ok
    assert p(None, None, None, f, f, 1, 0, 0, 4, 128, 64, 128, 0, 1.0, 1, 1, None, None, None, 0, None) == ok
    assert p(None, f, f, None, f, 1, 0, 9, 4, 128, 64, 128, 0, 1.0, 1, 1, None, None, None, 0, None) == bad
    assert p(None, f, f, f, f, 1, 8, 9, 4, 128, 64, 128, 8, 1.0, 1, 1, f, None, None, 0, None) == bad
    assert p(f, f, f, f, f, 1, 8, 9, 4, 128, 64, 128, 8, 1.0, 1, 1, None, None, None, 0, None) == bad
