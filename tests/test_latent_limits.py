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
