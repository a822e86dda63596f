"""Latent attention where its arithmetic is at its edges: keys that outweigh all others, rows without codes, queries that
are not finite, norms beyond fp32, empty calls, calls from two threads, and waits that run out."""
import pytest
import torch

import _latent_ref as L

pytestmark = pytest.mark.gpu
BF16, F32, I64, I32 = torch.bfloat16, torch.float32, torch.int64, torch.int32


@pytest.fixture(scope="module")
def C(gpu):
    import compressed_sparse_kv_csa_b200 as C
    C.csa_device_error()
    return C


def rng(seed):
    return torch.Generator().manual_seed(seed)


def ints(*v):
    return torch.tensor(v, dtype=I64, device="cuda")


def test_decode_contiguous_rows_and_pages_agree(C):
    """The same rows as one run and in pages of a tile: the same tiles, the same bits."""
    n = 128 * 300
    rows = C.KvRows.empty(n, 576, 64, "cuda")
    C.csa_quantize_kv((torch.randn((n, 576), generator=rng(1)) * torch.exp(torch.randn((n, 1), generator=rng(2)))).cuda(), rows)
    for H in (16, 64, 128):
        q = torch.randn((3, 1, H, 576), generator=rng(H)).to(BF16).cuda()
        pos = ints(12799, 12000, 12799)
        a = C.latent_attn_decode(q, rows, pos, 0.07, 12800, off=ints(0, 12800, 25600))
        b = C.latent_attn_decode(q, rows, pos, 0.07, 12800, pages=torch.arange(300, dtype=I32, device="cuda").view(3, 100), page_rows=128)
        assert torch.equal(a, b)
    assert C.csa_device_error() == 0
