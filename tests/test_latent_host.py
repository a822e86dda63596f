"""Latent attention without a GPU: the refusals of the C entry points and of the binding (which come
before anything is launched), the empty calls, and the identity that ties the two forms together."""
import ctypes

import pytest
import torch

import _latent_ref as L


@pytest.fixture(scope="module")
def C():
    import compressed_sparse_kv_csa_b200 as C
    return C


f = ctypes.c_void_p(0x100000)  # 16-byte aligned, never dereferenced
bad = ctypes.c_void_p(0x100004)


def kv(C, n=64, c=576, rd=64):
    return ctypes.byref(C._KvRows(0x100000, 0x200000, 0x300000, n, c, rd))


def test_append_refusals(C):
    def call(x=f, dt=0, n=4, g=f, eps=1e-6, base=1e4, pos=f, seq=None, B=4, pages=f, mp=2, pr=16, off=None, out=None):
        return C.lib().latent_append(x, dt, n, g, eps, base, pos, seq, B, pages, mp, pr, off, out or kv(C), None)
    I, U = C.CSA_ERR_INVALID_ARG, C.CSA_ERR_UNSUPPORTED
    assert call(x=None) == I and call(pos=None) == I and call(x=bad) == I and call(g=bad) == I
    assert call(dt=2) == I and call(n=-1) == I and call(B=-1) == I and call(B=3) == I
    assert call(pages=None) == I and call(mp=0) == I and call(pr=0) == I
    assert call(eps=-1.0) == I and call(eps=float("inf")) == I
    assert call(base=1.0) == I and call(base=-2.0) == I and call(base=float("inf")) == I and call(base=float("nan")) == I
    assert call(out=kv(C, rd=0)) == I and call(out=kv(C, c=64)) == I and call(out=kv(C, c=570)) == I
    assert call(out=kv(C, c=1024 + 16 + 64)) == U and call(out=kv(C, c=512 + 272, rd=272)) == U
    assert call(n=0) == C.CSA_OK and call(n=0, pages=None, off=f, g=None, base=0.0) == C.CSA_OK


def test_gather_refusals(C):
    def call(rows=None, cu=f, B=2, pages=f, mp=2, pr=16, off=None, n=8, lat=f, rope=f, dt=1):
        return C.lib().latent_gather(rows or kv(C), cu, None, B, pages, mp, pr, off, n, lat, rope, dt, None)
    I = C.CSA_ERR_INVALID_ARG
    assert call(cu=None) == I and call(B=-1) == I and call(n=-1) == I and call(lat=None, rope=None) == I
    assert call(lat=bad) == I and call(rope=bad) == I and call(dt=3) == I and call(pages=None) == I and call(pr=0) == I
    assert call(rows=kv(C, rd=0)) == I and call(rows=kv(C, c=2048)) == C.CSA_ERR_UNSUPPORTED
    assert call(n=(1 << 36) + 1) == C.CSA_ERR_UNSUPPORTED
    assert call(n=0) == C.CSA_OK and call(B=0) == C.CSA_OK


def test_decode_refusals(C):
    size = C.latent_attn_decode_workspace_size
    assert size(2, 1, 16, 512, 100) > 0 and size(0, 1, 16, 512, 100) == 0

    def call(q=f, rows=None, pos=f, pages=f, mp=2, pr=16, off=None, scale=1.0, B=2, Lq=1, H=16, ml=100, o=f, ws=f, n=1 << 30):
        return C.lib().latent_attn_decode(q, rows or kv(C), pos, pages, mp, pr, off, scale, B, Lq, H, ml, o, None, ws, n, None)
    I, U = C.CSA_ERR_INVALID_ARG, C.CSA_ERR_UNSUPPORTED
    assert call(q=None) == I and call(pos=None) == I and call(o=None) == I and call(q=bad) == I and call(o=bad) == I
    assert call(B=-1) == I and call(Lq=0) == I and call(H=0) == I and call(ml=-1) == I
    assert call(scale=float("nan")) == I and call(scale=float("inf")) == I
    assert call(pages=None) == I and call(mp=0) == I and call(pr=0) == I and call(rows=kv(C, rd=0)) == I
    assert call(H=129) == U and call(Lq=65) == U and call(ml=(1 << 30) + 1) == U and call(B=(1 << 18) + 1) == U
    assert call(rows=kv(C, c=640 + 64)) == U and call(rows=kv(C, c=48 + 64)) == U and call(rows=kv(C, c=512 + 144, rd=144)) == U
    assert call(ws=None) == C.CSA_ERR_WORKSPACE and call(n=size(2, 1, 16, 512, 100) - 1) == C.CSA_ERR_WORKSPACE
    assert call(B=0, ws=None) == C.CSA_OK


def test_prefill_refusals(C):
    def call(q=f, kv=f, kr=f, cq=f, ck=f, B=2, Tq=8, Tk=8, H=4, dn=128, dr=64, dv=128, mq=8, scale=1.0, dt=1, o=f):
        return C.lib().latent_attn_prefill(q, kv, kr, cq, ck, B, Tq, Tk, H, dn, dr, dv, mq, scale, 1, dt, o, None, None, 0, None)
    I, U = C.CSA_ERR_INVALID_ARG, C.CSA_ERR_UNSUPPORTED
    for k in ("q", "kv", "kr", "cq", "ck", "o"):
        assert call(**{k: None}) == I
    for k in ("q", "kv", "kr", "o"):
        assert call(**{k: bad}) == I
    for k in ("B", "Tq", "Tk", "mq", "H", "dn", "dr", "dv"):
        assert call(**{k: -1}) == I
    assert call(H=0) == I and call(dn=0) == I and call(dr=0) == I and call(dv=0) == I and call(dt=2) == I
    assert call(scale=float("nan")) == I
    assert call(H=129) == U and call(dn=120) == U and call(dr=24) == U and call(dv=272) == U and call(dn=208) == U
    assert call(Tq=1 << 31) == U and call(Tk=1 << 31) == U
    assert call(B=0) == C.CSA_OK and call(Tq=0) == C.CSA_OK and call(mq=0) == C.CSA_OK
    assert call(Tq=0, Tk=0, kv=None, kr=None) == C.CSA_OK


def test_prefill_workspace(C):
    size = C.latent_attn_prefill_workspace_size
    one = size(1, 1, 65536, 1, 128, 64, 128, 1)
    assert one > 0 and size(1, 256, 65536, 1, 128, 64, 128, 256) == one  # by blocks of 256 queries
    assert size(1, 256, 500, 1, 128, 64, 128, 256) == 0                  # keys too few to split
    assert size(1, 65536, 65536, 128, 128, 64, 128, 65536) == 0          # blocks enough
    assert size(1, 1, 65536, 1, 64, 64, 128, 1) == 0 and size(1, 1, 65536, 1, 128, 64, 128, 1, torch.float32) == 0
    assert size(0, 1, 65536, 1, 128, 64, 128, 1) == 0 and size(1, 1, -5, 1, 128, 64, 128, 1) == 0
    assert size(2 ** 40, 1, 2 ** 50, 1, 128, 64, 128, 1) == 0 and size(1, 2 ** 62, 65536, 128, 128, 64, 128, 2 ** 62) == 0
    assert size(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 128, 128, 64, 128, 2 ** 31 - 1) == 0


def test_binding_refuses_operands_it_would_misread(C):
    rows = C.KvRows.empty(64, 576, 64, "cpu")
    pages = torch.zeros((2, 4), dtype=torch.int32)
    pos = torch.zeros((2,), dtype=torch.int64)
    q = torch.zeros((2, 1, 16, 576), dtype=torch.bfloat16)
    x = torch.zeros((2, 576))
    go = dict(pages=pages, page_rows=16)
    with pytest.raises(ValueError):
        C.latent_append(x[:, :570], pos, rows, **go)
    with pytest.raises(ValueError):
        C.latent_append(torch.zeros((2, 1152))[:, ::2], pos, rows, **go)
    with pytest.raises(TypeError):
        C.latent_append(x.half(), pos, rows, **go)
    with pytest.raises(TypeError):
        C.latent_append(x, pos.int(), rows, **go)
    with pytest.raises(TypeError):
        C.latent_append(x, pos, rows, seq=pos, **go)
    with pytest.raises(ValueError):
        C.latent_append(x, pos, rows)
    with pytest.raises(ValueError):
        C.latent_append(x, pos, rows, off=pos, **go)
    with pytest.raises(TypeError):
        C.latent_attn_decode(q.float(), rows, pos, 1.0, 64, **go)
    with pytest.raises(ValueError):
        C.latent_attn_decode(q[..., :512], rows, pos, 1.0, 64, **go)
    with pytest.raises(ValueError):
        C.latent_attn_decode(q[:1], rows, pos[:1], 1.0, 64, **go)
    with pytest.raises(ValueError):
        C.latent_attn_decode(q, C.KvRows(rows.fp8, rows.rope[:32], rows.scale), pos, 1.0, 64, **go)
    with pytest.raises(ValueError, match="GPU"):
        C.latent_attn_decode(q, rows, pos, 1.0, 64, **go)
    with pytest.raises(ValueError):
        C.latent_gather(rows, torch.zeros((3,), dtype=torch.int64), **go)
    with pytest.raises(ValueError):
        C.latent_gather(rows, torch.zeros((2,), dtype=torch.int64), n=4, **go)
    cu = torch.zeros((3,), dtype=torch.int64)
    with pytest.raises(ValueError):
        C.latent_attn_prefill(torch.zeros((4, 2, 64)), torch.zeros((4, 2, 0)), torch.zeros((4, 64)), cu, cu, 4, 1.0)
    with pytest.raises(TypeError):
        C.latent_attn_prefill(torch.zeros((4, 2, 192)), torch.zeros((4, 2, 256), dtype=torch.bfloat16), torch.zeros((4, 64)), cu, cu, 4, 1.0)
    with pytest.raises(ValueError):
        C.latent_attn_prefill(torch.zeros((4, 2, 192)), torch.zeros((4, 3, 256)), torch.zeros((4, 64)), cu, cu, 4, 1.0)
    with pytest.raises(ValueError):
        C.latent_attn_prefill(torch.zeros((4, 2, 192)), torch.zeros((4, 2, 256)), torch.zeros((5, 64)), cu, cu, 4, 1.0)
    with pytest.raises(ValueError):
        C.latent_attn_prefill(torch.zeros((4, 2, 192)), torch.zeros((4, 2, 256)), torch.zeros((4, 64)), cu, cu[:2], 4, 1.0)


def test_forms_agree():
    """With k_nope = U lat and v = W lat, q.k = (q_nope U).lat + q_rope.rope and sum p v = W (sum p lat):
    the absorbed form of the reference equals the expanded one."""
    g = torch.Generator().manual_seed(1)
    n, H, R, rd, dn, dv = 37, 3, 64, 16, 32, 48
    lat, rope = torch.randn((n, R), generator=g, dtype=L.F64), torch.randn((n, rd), generator=g, dtype=L.F64)
    U, W = torch.randn((H, dn, R), generator=g, dtype=L.F64) / 8, torch.randn((H, dv, R), generator=g, dtype=L.F64) / 8
    q = torch.randn((n, H, dn + rd), generator=g, dtype=L.F64)
    kv = torch.cat([torch.einsum("hdr,nr->nhd", U, lat), torch.einsum("hdr,nr->nhd", W, lat)], 2)
    o, lse, *_ = L.prefill(q, kv, rope, [0, n], [0, n], dn, 0.2, True)
    qa = torch.cat([torch.einsum("nhd,hdr->nhr", q[..., :dn], U), q[..., dn:]], 2)[None]  # Lq = n tokens from position 0
    oa, la, *_ = L.decode(qa, lat, rope, lambda b, s: s, [0], 0.2, n)
    torch.testing.assert_close(torch.einsum("hdr,nhr->nhd", W, oa[0]), o, rtol=1e-10, atol=1e-10)
    torch.testing.assert_close(la[0], lse, rtol=1e-10, atol=1e-10)
