"""Latent attention where its arithmetic is at its edges: keys that outweigh all others, rows without codes, queries that
are not finite, norms beyond fp32, empty calls, calls from two threads, and waits that run out."""
import threading

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


# ------------------------------------------------------------------------------------------
# keys that outweigh the others
# ------------------------------------------------------------------------------------------

def check_weights(C, lat, score, H, R=512, B=160, lat_q=2.0 ** -10, pages=False, turn=False):
    """Decode of B sequences that all attend the rows (lat, and a score that the first rotated channel carries), with
    queries whose latent part is small, against the formula: one sequence lies in a CTA or two, so that a CTA walks through
    every kind of tile.  A sum over weights w = p * scale is held to 2^-8 of every term, or 2^-8 of the
    weighted mean of the rows' largest entries (include/csa.h); scores are sums of R + 64 products in fp32."""
    n = len(lat)
    x = torch.cat([lat, torch.zeros((n, 64))], 1)
    x[:, R] = score
    rows = C.KvRows.empty(n, R + 64, 64, "cuda")
    C.csa_quantize_kv(x.cuda(), rows)
    q = torch.randn((1, 1, H, R + 64), generator=rng(7)) * lat_q
    q[..., R:] = 0
    q[..., R] = -1.0 if turn else 1.0
    q = q.to(BF16).cuda()
    scale = -1.0 if turn else 1.0
    kw = dict(off=torch.zeros((B,), dtype=I64, device="cuda"))
    if pages:
        assert n % 128 == 0
        kw = dict(pages=torch.arange(n // 128, dtype=I32, device="cuda").repeat(B, 1), page_rows=128)
    pos = torch.full((B,), n - 1, dtype=I64, device="cuda")
    lse = torch.empty((B, 1, H), device="cuda")
    o = C.latent_attn_decode(q.expand(B, -1, -1, -1).contiguous(), rows, pos, scale, n, lse=lse, **kw)
    assert C.csa_device_error() == 0
    l, r = (t.cuda() for t in L.dequant(rows.fp8, rows.rope, rows.scale))
    key, qd = torch.cat([l, r], 1), q[0, 0].to(L.F64)
    z = qd @ key.T * scale
    ref_lse = z.logsumexp(1)
    p = (z - ref_lse[:, None]).exp()
    ref, size, top = p @ l, p @ l.abs(), p @ l.abs().amax(1)
    dz = (R + 64 + 8) * 2.0 ** -24 * (qd.abs() @ key.abs().T).amax(1)
    fp32 = 2 * dz + (n + 8) * 2.0 ** -24 + 2.0 ** -20
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + fp32)[:, None] * size + 2.0 ** -8 * top[:, None] + 1e-30
    err = (o[:, 0].to(L.F64) - ref).abs()
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    assert (err <= tol).all(), (float((err / tol).max()), float(err.norm() / ref.norm() / B ** 0.5))
    assert ((lse[:, 0].to(L.F64) - ref_lse).abs() <= dz + (n + 8) * 2.0 ** -24 + 2.0 ** -19 + 2.0 ** -22 * ref_lse.abs()).all()
    return ref, p


def values(n, R=512, seed=1, mean=1.0, std=0.1):
    return mean + std * torch.randn((n, R), generator=rng(seed))


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("first,middle", [(11.5, 7.25), (12.0, 6.75), (11.0, 7.75), (12.0, 0.0), (16.0, 9.0)])
def test_decode_small_weights_beside_a_heavy_key(C, H, first, middle):
    """A first key far above the rest, then a key in 128 that is above its neighbours: what the neighbours add up to (up to
    12% of the sum here) is held to the same bound as any."""
    n = 16384
    score = torch.zeros((n,))
    score[5::128] = middle
    score[0] = first
    _, p = check_weights(C, values(n), score, H)
    light = p[:, score == 0].sum(1)
    if first < 16:
        assert (light > 0.025).all()  # dropping them would be seen


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("std", [0.0, 1.0, 3.0])
def test_decode_spread_scores(C, H, std):
    n = 8192
    check_weights(C, values(n, std=1.0, mean=0.3), std * torch.randn((n,), generator=rng(3)), H, pages=True)


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("slope", [-0.004, 0.004])
def test_decode_scores_that_fall_or_rise(C, H, slope):
    n = 8192
    check_weights(C, values(n), torch.arange(n) * slope, H, pages=True, turn=True)


@pytest.mark.parametrize("H", [16, 64, 7])
@pytest.mark.parametrize("at,score", [([2], 12.0), ([2, 3, 200, 3999], 12.0), ([0], 60.0), (list(range(0, 4000, 3)), 20.0), ([3000], 90.0)])
@pytest.mark.parametrize("pages", [False, True])
def test_decode_heavy_keys_without_a_value(C, H, at, score, pages):
    """Keys whose latent part is zero (stored with a scale of 1) take their share of the sum of weights and leave the others'
    outputs as exact as without them."""
    n = 4096
    lat = values(n, mean=0.0, std=1.0)
    s = torch.zeros((n,))
    lat[at], s[at] = 0.0, score
    check_weights(C, lat, s, H, lat_q=2.0 ** -6, pages=pages)


@pytest.mark.parametrize("H", [16, 64])
def test_decode_rows_of_minus_zeros(C, H):
    """Rows without a value that hold codes of -0 (as +0) and a scale of 1."""
    n, B = 1000, 160
    rows = C.KvRows.empty(n, 576, 64, "cuda")
    x = torch.randn((n, 576), generator=rng(4))
    x[:, 512:] = 0
    x[3::7, 512] = 12.0
    C.csa_quantize_kv(x.cuda(), rows)
    rows.fp8[3::7] = torch.where(torch.rand((n, 512), generator=rng(5)).cuda() < 0.5, 0x80, 0).to(torch.uint8)[3::7]
    rows.scale[3::7] = 1.0
    q = torch.zeros((B, 1, H, 576), dtype=BF16, device="cuda")
    q[..., 512] = 1.0
    q[..., :512] = torch.randn((H, 512), generator=rng(6)).cuda() * 2.0 ** -6
    o = C.latent_attn_decode(q, rows, torch.full((B,), n - 1, dtype=I64, device="cuda"), 1.0, n, off=torch.zeros((B,), dtype=I64, device="cuda"))
    l, r = (t.cuda() for t in L.dequant(rows.fp8, rows.rope, rows.scale))
    qd, key = q[0, 0].to(L.F64), torch.cat([l, r], 1)
    p = (qd @ key.T).softmax(1)
    # as above
    fp32 = 2 * (576 + 8) * 2.0 ** -24 * (qd.abs() @ key.abs().T).amax(1) + (n + 8) * 2.0 ** -24 + 2.0 ** -20
    tol = 2.0 ** -8 * (p @ l).abs() + (2.0 ** -8 + fp32)[:, None] * (p @ l.abs()) + 2.0 ** -8 * (p @ l.abs().amax(1))[:, None]
    assert ((o[:, 0].to(L.F64) - p @ l).abs() <= tol).all()


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("code", [0x7e, 0x01, 0x81])
def test_decode_rows_of_one_code(C, H, code):
    """A scale of 1 and one code, in any channel, the largest or the smallest there is: a row with a value.  With w = 2^x the
    one weight, the output is (w rounded) code / w: w lies in 4 .. 8, is off by at most 2^-8 of itself and divided by
    itself as it was, so the output by that and its own half step, 2^-8; the other channels are 0."""
    rows = C.KvRows.empty(512, 576, 64, "cuda")
    rows.fp8.zero_(), rows.rope.zero_(), rows.scale.fill_(1.0)
    rows.fp8.fill_diagonal_(code)
    q = torch.randn((512, 1, H, 576), generator=rng(1)).to(BF16).cuda()
    o = C.latent_attn_decode(q, rows, torch.zeros((512,), dtype=I64, device="cuda"), 0.05, 1, off=torch.arange(512, device="cuda"))
    want = torch.zeros((512, 512), dtype=torch.float64)
    want.fill_diagonal_(float(torch.tensor([code], dtype=torch.uint8).view(torch.float8_e4m3fn).double()))
    assert ((o[:, 0].cpu().double() - want[:, None]).abs() <= 2.02 * 2.0 ** -8 * want[:, None].abs()).all() and C.csa_device_error() == 0


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("size", [2.0 ** 4, 2.0 ** 8, 2.0 ** 12])
def test_decode_queries_with_an_outlier(C, H, size):
    """One channel of the queries far above the others, where the keys have nothing: the others count to 2^-18 of it
    (include/csa.h), which a score's error adds up over a key's channels."""
    n = 3000
    x = torch.randn((n, 576), generator=rng(1))
    x[:, 5] = 0
    rows = C.KvRows.empty(n, 576, 64, "cuda")
    C.csa_quantize_kv(x.cuda(), rows)
    q = torch.randn((1, 1, H, 576), generator=rng(2))
    q[..., 5] = size
    q = q.to(BF16).cuda()
    lse = torch.empty((1, 1, H), device="cuda")
    o = C.latent_attn_decode(q, rows, ints(n - 1), 0.05, n, off=ints(0), lse=lse)
    l, r = (t.cuda() for t in L.dequant(rows.fp8, rows.rope, rows.scale))
    key, qd = torch.cat([l, r], 1), q[0, 0].to(L.F64)
    z = qd @ key.T * 0.05
    p = z.softmax(1)
    dz = 0.05 * ((576 + 8) * 2.0 ** -24 * (qd.abs() @ key.abs().T).amax(1) + 2.0 ** -18 * size * l.abs().sum(1).max())
    tol = 2.0 ** -8 * (p @ l).abs() + (2 * dz + 2.0 ** -8 + (n + 8) * 2.0 ** -24 + 2.0 ** -20)[:, None] * (p @ l.abs()) + 2.0 ** -8 * (p @ l.abs().amax(1))[:, None]
    assert ((o[0, 0].to(L.F64) - p @ l).abs() <= tol).all() and C.csa_device_error() == 0
    assert ((lse[0, 0].to(L.F64) - z.logsumexp(1)).abs() <= dz + (n + 8) * 2.0 ** -24 + 2.0 ** -19).all()


# ------------------------------------------------------------------------------------------
# numbers that are not finite, or beyond fp32 on the way
# ------------------------------------------------------------------------------------------

BAD = [float("nan"), float("inf"), -float("inf")]


@pytest.mark.parametrize("R,rd,H", [(512, 64, 8), (512, 64, 40), (256, 64, 8), (96, 16, 3)])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("n", [1, 40, 3000])
def test_decode_of_a_query_that_is_not_finite(C, R, rd, H, bad, n):
    """It makes NaN of its own row, as the formula does, and not the zeros of a row that sees nothing."""
    rows = C.KvRows.empty(n, R + rd, rd, "cuda")
    x = torch.randn((n, R + rd), generator=rng(1))
    x[0, 3] = 1.0 if bad > 0 else -1.0  # (one key alone: a score of +inf, whose softmax is inf / inf)
    C.csa_quantize_kv(x.cuda(), rows)
    q = torch.randn((2, 1, H, R + rd), generator=rng(2)).to(BF16).cuda()
    pos, off = ints(n - 1, n - 1), ints(0, 0)
    lse = torch.empty((2, 1, H), device="cuda")
    good = C.latent_attn_decode(q, rows, pos, 0.05, n, off=off)
    q[1, 0, H // 2, 3] = bad
    o = C.latent_attn_decode(q, rows, pos, 0.05, n, off=off, lse=lse)
    hit = torch.zeros((2, 1, H), dtype=torch.bool, device="cuda")
    hit[1, 0, H // 2] = True
    assert torch.equal(o[~hit], good[~hit]) and torch.isfinite(lse[~hit]).all()
    assert o[hit].isnan().all() and lse[hit].isnan().all()


@pytest.mark.parametrize("dims,dtype", [((128, 64, 128), BF16), ((128, 64, 128), F32), ((64, 32, 96), BF16)])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("n", [1, 40, 300])
def test_prefill_of_a_query_that_is_not_finite(C, dims, dtype, bad, n):
    dn, dr, dv = dims
    q, kv, kr = (torch.randn(s, generator=rng(i)).to(dtype).cuda() for i, s in enumerate(((n, 2, dn + dr), (n, 2, dn + dv), (n, dr))))
    kv[0, :, 3] = 1.0 if bad > 0 else -1.0
    cu = ints(0, n)
    lse = torch.empty((n, 2), device="cuda")
    good = C.latent_attn_prefill(q, kv, kr, cu, cu, n, 0.1)
    q[n // 2, 1, 3] = bad
    o = C.latent_attn_prefill(q, kv, kr, cu, cu, n, 0.1, lse=lse)
    hit = torch.zeros((n, 2), dtype=torch.bool, device="cuda")
    hit[n // 2, 1] = True
    assert torch.equal(o[~hit], good[~hit]) and torch.isfinite(lse[~hit]).all()
    assert o[hit].isnan().all() and lse[hit].isnan().all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R", [512, 1024, 32])
@pytest.mark.parametrize("eps", [1e-6, 0.0, 2.0 ** -120])
@pytest.mark.parametrize("n", [1, 2600])
def test_append_norms_beyond_fp32(C, dtype, R, eps, n):
    """Rows whose squares overflow fp32, or underflow where eps does not cover it, between ordinary ones: their norm is
    that of the formula.  Off by at most 32 half steps of fp32, as any row's; a code by half a step of E4M3."""
    sizes = torch.tensor([1.0, 1e17, 1e20, 3e37, 1e-3, 1e-20, 1e-30, 1e-36])[torch.arange(n) * 5 % 8 if n > 1 else torch.tensor([3])]
    x = (torch.randn((n, R + 64), generator=rng(R)) * sizes[:, None]).to(dtype)
    gain = 1 + 0.2 * torch.randn((R,), generator=rng(1))
    out = C.KvRows.empty(n, R + 64, 64, "cuda")
    C.latent_append(x.cuda(), torch.zeros((n,), dtype=I64, device="cuda"), out, g=gain.cuda(), eps=eps, off=torch.arange(n, device="cuda"))
    assert C.csa_device_error() == 0
    lat, _ = L.append_rows(x, torch.zeros((n,), dtype=I64), R, gain, float(torch.tensor(eps, dtype=F32)))
    got, _ = L.dequant(out.fp8, out.rope, out.scale)
    e = 32 * 2.0 ** -24
    want = lat.abs().amax(1) / 448
    sc = out.scale.cpu().to(L.F64)
    assert ((sc - want).abs() <= 2 * e * want + 2.0 ** -149).all()
    tol = lat.abs() * (2.0 ** -4 + 4 * e) + sc[:, None] * 2.0 ** -10 + 448 * 2.0 ** -149
    assert ((got - lat).abs() <= tol).all()


# ------------------------------------------------------------------------------------------
# calls
# ------------------------------------------------------------------------------------------

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


# ------------------------------------------------------------------------------------------
# waits that run out
# ------------------------------------------------------------------------------------------

def runs_out(C, call, path):
    """With a limit of 1 ns every wait that has it is one test that gives up: the kernel reports it and winds down, its own
    copies and MMAs waited for (the warps without it take 2 s to give up).  Nothing faults or hangs, and the next calls
    are as before."""
    want = call()
    assert C.csa_last_path() == path and C.csa_device_error() == 0
    prev = C.csa_set_wait_limit_ns(1)
    try:
        call()
        torch.cuda.synchronize()
        err = C.csa_device_error()
    finally:
        assert C.csa_set_wait_limit_ns(prev) == 1
    assert err & C.CSA_DEVERR_TIMEOUT
    for _ in range(2):
        assert torch.equal(call(), want)
    assert C.csa_device_error() == 0


@pytest.mark.parametrize("H,page", [(16, 128), (64, 32), (16, 1), (64, 0)])
def test_decode_waits_run_out(C, H, page):
    n, B = 1000, 160  # more tiles a CTA than stages, and one that is partly seen
    rows = C.KvRows.empty(1024, 576, 64, "cuda")
    C.csa_quantize_kv(torch.randn((1024, 576), generator=rng(1)).cuda(), rows)
    q = torch.randn((B, 1, H, 576), generator=rng(2)).to(BF16).cuda()
    pos = torch.full((B,), n - 1, dtype=I64, device="cuda")
    kw = dict(pages=torch.arange(1024 // page, dtype=I32, device="cuda").repeat(B, 1), page_rows=page) if page else dict(off=torch.zeros_like(pos))
    runs_out(C, lambda: C.latent_attn_decode(q, rows, pos, 0.05, n, **kw), C.CSA_PATH_LATENT_DECODE_TC)


@pytest.mark.parametrize("nq,nk,H", [(700, 700, 2), (1, 5, 1), (300, 4100, 2)])
def test_prefill_waits_run_out(C, nq, nk, H):
    q, kv, kr = (torch.randn(s, generator=rng(i)).to(BF16).cuda() for i, s in enumerate(((nq, H, 192), (nk, H, 256), (nk, 64))))
    cq, ck = ints(0, nq), ints(0, nk)
    runs_out(C, lambda: C.latent_attn_prefill(q, kv, kr, cq, ck, nq, 0.1), C.CSA_PATH_LATENT_PREFILL_TC)


@pytest.mark.parametrize("page_rows", [2 ** 31 - 128, 2 ** 31 - 1, 2 ** 30 + 128])
def test_one_page_larger_than_any_cache(C, page_rows):
    """A page size that no cache reaches: all of a sequence's rows are in its first page."""
    n = 1024
    rows, flat = (C.KvRows.empty(n, 576, 64, "cuda") for _ in range(2))
    x = torch.randn((n, 576), generator=rng(1)).cuda()
    pos, seq = torch.arange(n, device="cuda"), torch.zeros((n,), dtype=I32, device="cuda")
    pages = torch.zeros((1, 1), dtype=I32, device="cuda")
    C.latent_append(x, pos, rows, seq=seq, pages=pages, page_rows=page_rows)
    C.latent_append(x, pos, flat, seq=seq, off=ints(0))
    assert torch.equal(rows.fp8, flat.fp8) and torch.equal(rows.scale, flat.scale)
    for H in (16, 64):
        q = torch.randn((1, 1, H, 576), generator=rng(2)).to(BF16).cuda()
        a = C.latent_attn_decode(q, rows, ints(n - 1), 0.07, n, pages=pages, page_rows=page_rows)
        assert torch.equal(a, C.latent_attn_decode(q, rows, ints(n - 1), 0.07, n, off=ints(0)))
    a, b = C.latent_gather(rows, ints(0, n), n=n, pages=pages, page_rows=page_rows), C.latent_gather(rows, ints(0, n), n=n, off=ints(0))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert C.csa_device_error() == 0


def test_two_threads_with_different_channel_counts(C):
    """Calls of two host threads on streams of their own do not take each other's shared memory limit."""
    cases, failed = [], []
    for R, rd in ((512, 128), (32, 16)):
        rows = C.KvRows.empty(64, R + rd, rd, "cuda")
        C.csa_quantize_kv(torch.randn((64, R + rd), generator=rng(R)).cuda(), rows)
        q = torch.randn((1, 1, 4, R + rd), generator=rng(1)).to(BF16).cuda()
        d = 32 if R == 512 else 256
        p = [torch.randn(s, generator=rng(i)).cuda() for i, s in enumerate(((8, 1, d), (8, 1, d - 16 + d), (8, 16)))]
        cases.append((rows, q, ints(63), ints(0), p, ints(0, 8)))

    def work(rows, q, pos, off, p, cu):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                want = C.latent_attn_decode(q, rows, pos, 0.1, 64, off=off), C.latent_attn_prefill(*p, cu, cu, 8, 0.1)
                for _ in range(400):
                    got = C.latent_attn_decode(q, rows, pos, 0.1, 64, off=off), C.latent_attn_prefill(*p, cu, cu, 8, 0.1)
                s.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, want))
        except Exception as e:
            failed.append(e)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=c) for c in cases]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed, failed[0]


# ------------------------------------------------------------------------------------------
# calls
# ------------------------------------------------------------------------------------------

def test_empty_calls(C):
    """No rows, no sequences, no queries: nothing to do, and nothing wrong."""
    rows = C.KvRows.empty(32, 576, 64, "cuda")
    pages, none = torch.zeros((0, 2), dtype=I32, device="cuda"), torch.zeros((0,), dtype=I64, device="cuda")
    one = torch.zeros((1, 2), dtype=I32, device="cuda")
    x = torch.zeros((0, 576), device="cuda")
    C.latent_append(x, none, rows, g=torch.ones((512,), device="cuda"), base=10000.0, pages=one, page_rows=16)
    C.latent_append(x, none, rows, seq=torch.zeros((0,), dtype=I32, device="cuda"), off=none)
    C.latent_append(x, none, rows, pages=pages, page_rows=16)
    lat, rope = C.latent_gather(rows, ints(0), n=0, pages=pages, page_rows=16)
    assert lat.shape == (0, 512) and rope.shape == (0, 64)
    lat, _ = C.latent_gather(rows, ints(0, 0), n=0, off=ints(0))
    assert lat.shape == (0, 512)
    lat = torch.full((3, 512), 7.0, device="cuda")
    C.latent_gather(rows, ints(0), off=none, lat=lat)
    assert (lat == 7).all()
    o = C.latent_attn_decode(torch.zeros((0, 1, 16, 576), dtype=BF16, device="cuda"), rows, none, 1.0, 64, pages=pages, page_rows=16)
    assert o.shape == (0, 1, 16, 512)
    for dt in (BF16, F32):
        e = lambda *s: torch.zeros(s, dtype=dt, device="cuda")
        assert C.latent_attn_prefill(e(0, 4, 192), e(0, 4, 256), e(0, 64), ints(0), ints(0), 0, 1.0).shape == (0, 4, 128)
        assert C.latent_attn_prefill(e(0, 4, 192), e(9, 4, 256), e(9, 64), ints(0, 0), ints(0, 9), 0, 1.0).shape == (0, 4, 128)
        o, lse = torch.full((3, 4, 128), 7.0, dtype=dt, device="cuda"), torch.full((3, 4), 7.0, device="cuda")
        C.latent_attn_prefill(e(3, 4, 192), e(0, 4, 256), e(0, 64), ints(0, 3), ints(0, 0), 3, 1.0, o=o, lse=lse)
        assert (o == 0).all() and (lse == -torch.inf).all()  # queries without keys
    assert C.csa_device_error() == 0


def test_decode_of_many_sequences(C):
    """More sequences than SMs and warps, of 0 to 300 keys: each as by itself."""
    B, H = 2000, 16
    rows = C.KvRows.empty(4096, 576, 64, "cuda")
    C.csa_quantize_kv(torch.randn((4096, 576), generator=rng(1)).cuda(), rows)
    q = torch.randn((B, 1, H, 576), generator=rng(2)).to(BF16).cuda()
    lens = torch.randint(0, 301, (B,), generator=rng(3)).cuda()
    off = torch.randint(0, 3700, (B,), generator=rng(4)).cuda()
    lse = torch.empty((B, 1, H), device="cuda")
    o = C.latent_attn_decode(q, rows, lens - 1, 0.07, 300, off=off, lse=lse)
    assert C.csa_device_error() == 0
    l, r = (t.cuda() for t in L.dequant(rows.fp8, rows.rope, rows.scale))
    at = off[:, None] + torch.arange(300, device="cuda")
    key, v = torch.cat([l, r], 1)[at], l[at]
    z = torch.einsum("bhc,bsc->bhs", q[:, 0].to(L.F64), key) * 0.07
    z = z.masked_fill((torch.arange(300, device="cuda") >= lens[:, None])[:, None], -torch.inf)
    some = lens > 0
    p = z[some].softmax(2)
    ref, size = p @ v[some], p @ v[some].abs()
    dz = (576 + 8) * 2.0 ** -24 * 0.07 * torch.einsum("bhc,bsc->bhs", q[:, 0].to(L.F64).abs(), key.abs()).amax(2)[some]
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * dz + 308 * 2.0 ** -24 + 2.0 ** -20)[..., None] * size + 2.0 ** -8 * (p @ v[some].abs().amax(2, keepdim=True))
    assert ((o[some, 0].to(L.F64) - ref).abs() <= tol).all()
    assert (o[~some] == 0).all() and (lse[~some] == -torch.inf).all()
    ref = z[some].logsumexp(2)
    assert ((lse[some, 0].to(L.F64) - ref).abs() <= dz + 308 * 2.0 ** -24 + 2.0 ** -19 + 2.0 ** -22 * ref.abs()).all()
