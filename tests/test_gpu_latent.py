"""Latent attention on the GPU against the 64-bit formulas: latent_append, latent_gather,
latent_attn_decode (absorbed form) and latent_attn_prefill (expanded form), at the sizes and masks where
they can go wrong, and the four together as a layer uses them."""
import numpy as np
import pytest
import torch

import _latent_ref as L

pytestmark = pytest.mark.gpu
BF16, F32, I64, I32, I16 = torch.bfloat16, torch.float32, torch.int64, torch.int32, torch.int16
V_STEP = 2.0 ** -8  # half a step of the decode kernel's probabilities: 8 bits in two terms of 4 (on the tensor cores)
NAN8 = 0x7f            # the E4M3 code of NaN


@pytest.fixture(scope="module")
def C(gpu):
    import compressed_sparse_kv_csa_b200 as C
    C.csa_device_error()
    return C


def rng(seed):
    return torch.Generator().manual_seed(seed)


def ints(*v):
    return torch.tensor(v, dtype=I64, device="cuda")


def cache(C, n, R, rd, seed=0, spread=0.0):
    """n rows ~ N(0, 1), their sizes spread by e^(spread N(0, 1)), quantised as the library quantises."""
    g = rng(seed)
    x = torch.randn((n, R + rd), generator=g)
    x[:, :R] *= torch.exp(spread * torch.randn((n, 1), generator=g))
    rows = C.KvRows.empty(n, R + rd, rd, "cuda")
    C.csa_quantize_kv(x.cuda(), rows)
    return rows


def poison(rows, keep):
    """NaN in every row that is not in `keep`."""
    m = torch.ones((rows.n,), dtype=torch.bool)
    m[torch.tensor(sorted(keep), dtype=torch.long)] = False
    m = m.cuda()
    rows.fp8[m] = NAN8
    rows.rope[m] = float("nan")
    rows.scale[m] = float("nan")


def table(B, per, page_rows, seed=0, spare=1):
    """A shuffled page table [B, per] over (B * per + spare) pages, and the cache rows behind it."""
    n = B * per + spare
    return torch.randperm(n, generator=rng(seed))[:B * per].to(I32).view(B, per).cuda(), n * page_rows


# ------------------------------------------------------------------------------------------
# append
# ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("R,rd", [(512, 64), (32, 16), (240, 32), (1024, 256), (272, 96)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("norm,base", [(True, 10000.0), (False, 0.0), (True, 0.0), (False, 500000.0)])
def test_append(C, R, rd, dtype, norm, base):
    g = rng(R + rd)
    B, page, per = 5, 16, 9
    pages, rows_n = table(B, per, page, 3)
    n = 41
    x = (torch.randn((n, R + rd), generator=g) * torch.exp(2 * torch.randn((n, 1), generator=g))).to(dtype).cuda()
    x[7, :R] = 0
    x[8] = 0
    at = torch.randperm(B * per * page, generator=g)[:n]
    seq, pos = (at // (per * page)).to(I32).cuda(), (at % (per * page)).cuda()
    skipped = [0, 20]
    pos[skipped] = -1
    gain = (1 + 0.2 * torch.randn((R,), generator=g)).cuda() if norm else None
    out = cache(C, rows_n, R, rd)
    before = [t.clone() for t in (out.fp8, out.rope, out.scale)]
    C.latent_append(x, pos, out, g=gain, eps=1e-6, base=base, seq=seq, pages=pages, page_rows=page)
    assert C.csa_device_error() == 0
    lat, rope = L.append_rows(x, pos, R, gain, 1e-6, base)
    glat, grope = L.dequant(out.fp8, out.rope, out.scale)
    scale = out.scale.cpu().to(L.F64)
    written = []
    for i in range(n):
        if i in skipped:
            continue
        r = L.row_of(pages.cpu(), page, None, int(seq[i]), int(pos[i]))
        written.append(r)
        # the norm is off by at most 32 half steps of fp32: the sum of 1024 squares over 32 lanes, mean, root, two products
        e = 32 * 2.0 ** -24
        amax = lat[i].abs().max()
        want = amax / 448 if amax > 0 else torch.tensor(1.0, dtype=L.F64)
        assert abs(scale[r] - want) <= 2 * e * want
        # a code is the nearest value: half a step of E4M3 (2^-4 relative, 2^-10 of the scale below the smallest normal)
        tol = lat[i].abs() * (2.0 ** -4 + 4 * e) + scale[r] * 2.0 ** -10
        assert ((glat[r] - lat[i]).abs() <= tol).all()
        pair = x[i, R:].cpu().to(L.F64).view(-1, 2).norm(dim=1).repeat_interleave(2)
        assert ((grope[r] - rope[i]).abs() <= 2.0 ** -8 * rope[i].abs() + 2.0 ** -20 * pair).all()
    rest = torch.ones((rows_n,), dtype=torch.bool)
    rest[written] = False
    for t, b in zip((out.fp8, out.rope, out.scale), before):
        assert torch.equal(t[rest.cuda()], b[rest.cuda()])  # rows that the call does not name


def test_append_far_positions(C):
    """A rotation at position 2^31 + 5: the angle is formed in 64 bits.  exp and log of the frequency
    are off by a few 2^-53 of ln base / 1 < 16, the angle by 2^-48 of the position."""
    g = rng(5)
    pos = ints(2 ** 31 + 5, 2 ** 24 + 1, 1048576)
    x = torch.randn((3, 576), generator=g)
    out = C.KvRows.empty(3, 576, 64, "cuda")
    off = -pos + ints(0, 1, 2)
    C.latent_append(x.cuda(), pos, out, base=10000.0, off=off)
    assert C.csa_device_error() == 0
    _, rope = L.append_rows(x, pos, 512, None, 0, 10000.0)
    pair = x[:, 512:].to(L.F64).view(3, -1, 2).norm(dim=2).repeat_interleave(2, 1)
    tol = 2.0 ** -8 * rope.abs() + (2.0 ** -20 + 2.0 ** -48 * pos.cpu().to(L.F64)[:, None]) * pair
    assert ((out.rope.cpu().to(L.F64) - rope).abs() <= tol).all()


def test_append_equals_the_quantiser_and_one_row_at_a_time(C):
    """Without norm and rotation the rows are csa_quantize_kv's, bit for bit, in one call or many."""
    x = torch.randn((50, 576), generator=rng(2)).to(BF16).cuda()
    ref = C.KvRows.empty(50, 576, 64, "cuda")
    C.csa_quantize_kv(x, ref)
    off = torch.arange(50, device="cuda")
    zero = torch.zeros((50,), dtype=I64, device="cuda")
    a, b = C.KvRows.empty(50, 576, 64, "cuda"), C.KvRows.empty(50, 576, 64, "cuda")
    C.latent_append(x, zero, a, off=off)
    for i in range(50):
        C.latent_append(x[i:i + 1], zero[:1], b, off=off[i:i + 1].contiguous())
    for t in (a, b):
        assert torch.equal(t.fp8, ref.fp8) and torch.equal(t.rope, ref.rope) and torch.equal(t.scale, ref.scale)


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-8, 1.0, 3e30, 1e38])
@pytest.mark.parametrize("R", [512, 1024, 32])
def test_append_codes_are_those_of_the_division(C, size, R):
    """Rows whose entries lie on and beside the middles between codes, at scales down to where a reciprocal leaves
    fp32's range: bit for bit csa_quantize_kv's, which divides."""
    g = rng(11)
    n = 300
    x = torch.randn((n, R + 64), generator=g)
    mid = (torch.randint(0, 448 * 16, (n // 2, R), generator=g).float() + 0.5) / 16  # middles, over a scale of 1
    x[:n // 2, :R] = mid * torch.where(torch.rand((n // 2, R), generator=g) < 0.5, -1.0, 1.0)
    x[:n // 2, 3] = 448.0
    x = (x * size).cuda()
    ref, out = C.KvRows.empty(n, R + 64, 64, "cuda"), C.KvRows.empty(n, R + 64, 64, "cuda")
    C.csa_quantize_kv(x, ref)
    C.latent_append(x, torch.zeros((n,), dtype=I64, device="cuda"), out, off=torch.arange(n, device="cuda"))
    assert torch.equal(out.scale, ref.scale) and torch.equal(out.fp8, ref.fp8) and torch.equal(out.rope, ref.rope)


def test_append_many_rows(C):
    """More rows than warps: the same as a few at a time."""
    n = 50001
    x = torch.randn((n, 576), generator=rng(12)).to(BF16).cuda()
    pos, off = torch.arange(n, device="cuda"), torch.zeros((1,), dtype=I64, device="cuda")
    seq = torch.zeros((n,), dtype=I32, device="cuda")
    gain = (1 + 0.1 * torch.randn((512,), generator=rng(13))).cuda()
    a, b = C.KvRows.empty(n, 576, 64, "cuda"), C.KvRows.empty(n, 576, 64, "cuda")
    C.latent_append(x, pos, a, g=gain, base=10000.0, seq=seq, off=off)
    for i in range(0, n, 4000):
        C.latent_append(x[i:i + 4000], pos[i:i + 4000], b, g=gain, base=10000.0, seq=seq[i:i + 4000], off=off)
    assert torch.equal(a.fp8, b.fp8) and torch.equal(a.rope, b.rope) and torch.equal(a.scale, b.scale)


@pytest.mark.parametrize("R,rd", [(512, 64), (32, 16), (240, 32), (1024, 256), (272, 96)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("norm,base", [(True, 10000.0), (False, 0.0)])
@pytest.mark.parametrize("n", [2500, 5003])
def test_append_several_rows_a_warp(C, R, rd, dtype, norm, base, n):
    """Rows that a warp takes side by side, skipped, refused and odd ones among them: those of calls whose warps take one."""
    g = rng(n + R)
    x = (torch.randn((n, R + rd), generator=g) * 3).to(dtype).cuda()
    x[7, 5], x[11, 0], x[13, :R], x[14, :R], x[15, :R] = float("nan"), float("inf"), 0.0, 1e-38, 1e30
    pos = torch.randperm(n, generator=g).cuda()
    pos[3::97], pos[5::101] = -1, 1 << 40  # skipped, refused
    seq, off = torch.zeros((n,), dtype=I32, device="cuda"), ints(0)
    gain = (1 + 0.1 * torch.randn((R,), generator=g)).cuda() if norm else None
    a, b = C.KvRows.empty(n, R + rd, rd, "cuda"), C.KvRows.empty(n, R + rd, rd, "cuda")
    for t in (a, b):
        t.fp8.fill_(0x55), t.rope.fill_(7.0), t.scale.fill_(7.0)
    C.latent_append(x, pos, a, g=gain, base=base, seq=seq, off=off)
    assert C.csa_device_error() == C.CSA_DEVERR_INDEX
    for i in range(0, n, 500):
        C.latent_append(x[i:i + 500], pos[i:i + 500], b, g=gain, base=base, seq=seq[i:i + 500], off=off)
    assert C.csa_device_error() == C.CSA_DEVERR_INDEX
    assert torch.equal(a.fp8, b.fp8) and torch.equal(a.rope.view(I16), b.rope.view(I16)) and torch.equal(a.scale.view(I32), b.scale.view(I32))


def test_append_refused_rows(C):
    """A page outside the cache, a position behind the table and a sequence that is not there are refused,
    the other rows written."""
    x = torch.randn((5, 576), generator=rng(1)).cuda()
    out = C.KvRows.empty(32, 576, 64, "cuda")
    for t in (out.fp8, out.rope, out.scale):
        t.zero_()
    pages = torch.tensor([[1, 7], [0, -3]], dtype=I32, device="cuda")  # 2 pages of 16 rows exist
    seq = torch.tensor([0, 0, 1, 2, 1], dtype=I32, device="cuda")
    C.latent_append(x, ints(3, 16, 31, 0, 5), out, seq=seq, pages=pages, page_rows=16)
    assert C.csa_device_error() == C.CSA_DEVERR_INDEX
    assert out.scale.nonzero()[:, 0].tolist() == [5, 19]
    C.latent_append(x, ints(0, 0, 32, 0, 0), out, seq=torch.full((5,), -1, dtype=I32, device="cuda"), pages=pages, page_rows=16)
    assert C.csa_device_error() == C.CSA_DEVERR_INDEX
    assert out.scale.nonzero()[:, 0].tolist() == [5, 19]


# ------------------------------------------------------------------------------------------
# gather
# ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("R,rd", [(512, 64), (32, 16), (240, 32), (1024, 256)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("paged", [True, False])
def test_gather(C, R, rd, dtype, paged):
    lens, starts, page = [5, 0, 33, 1, 16, 0], [0, 9, 7, 40, 16, 3], 16
    cu = np.concatenate([[3], 3 + np.cumsum(lens)])
    pages, rows_n = table(6, 4, page, 1)
    off = ints(*[30 * b for b in range(6)])
    n_off = 30 * 6 + 60
    rows = cache(C, rows_n if paged else n_off, R, rd, 4, 1.0)
    kw = dict(pages=pages, page_rows=page) if paged else dict(off=off)
    n = int(cu[-1]) + 9
    lat, rope = torch.full((n, R), 7.0, dtype=dtype, device="cuda"), torch.full((n, rd), 7.0, dtype=dtype, device="cuda")
    C.latent_gather(rows, ints(*cu), start=ints(*starts), lat=lat, rope=rope, **kw)
    assert C.csa_device_error() == 0
    elat, erope = L.dequant(rows.fp8, rows.rope, rows.scale)
    at = [L.row_of(pages.cpu() if paged else None, page, off, b, s0 + j) for b, (s0, m) in enumerate(zip(starts, lens)) for j in range(m)]
    # codes times scale is exact in more than fp32: one rounding
    got = lat.cpu().to(L.F64)[3:cu[-1]]
    assert ((got - elat[at]).abs() <= L.STEP[dtype] * elat[at].abs()).all()
    assert torch.equal(rope.cpu().to(L.F64)[3:cu[-1]], erope[at])
    for t in (lat, rope):  # rows in front of the first run and behind the last
        assert (t[:3] == 7).all() and (t[int(cu[-1]):] == 7).all()
    only = torch.full((n, rd), 7.0, dtype=dtype, device="cuda")
    assert C.latent_gather(rows, ints(*cu), start=ints(*starts), rope=only, **kw)[0] is None
    assert torch.equal(only, rope)
    only = torch.full((n, R), 7.0, dtype=dtype, device="cuda")
    C.latent_gather(rows, ints(*cu), start=ints(*starts), lat=only, **kw)
    assert torch.equal(only, lat)
    short = torch.full((11, R), 7.0, dtype=dtype, device="cuda")  # fewer rows than the runs
    C.latent_gather(rows, ints(*cu), start=ints(*starts), lat=short, **kw)
    assert torch.equal(short, lat[:11])


def test_gather_refused_rows_are_zero(C):
    rows = cache(C, 32, 512, 64)
    pages = torch.tensor([[1, 7]], dtype=I32, device="cuda")
    lat, rope = C.latent_gather(rows, ints(0, 40), n=40, pages=pages, page_rows=16)
    assert C.csa_device_error() == C.CSA_DEVERR_INDEX
    assert (lat[:16].float().abs().sum(1) > 0).all() and (lat[16:] == 0).all() and (rope[16:] == 0).all()
    lat, _ = C.latent_gather(rows, ints(0, 4), n=4, start=ints(-2), pages=pages, page_rows=16)
    assert C.csa_device_error() == C.CSA_DEVERR_INDEX
    assert (lat[:2] == 0).all() and torch.equal(lat[2:], C.latent_gather(rows, ints(0, 2), n=2, pages=pages, page_rows=16)[0])


# ------------------------------------------------------------------------------------------
# decode
# ------------------------------------------------------------------------------------------

def run_decode(C, lens, H, Lq, R, rd, page, seed=0, spread=0.3, scale=None, max_len=None, q=None, rows=None):
    """A decode over sequences of `lens` positions (the new tokens included; less than Lq: padding in
    front), with NaN in every row that nobody sees, against the formula.  page 0: contiguous."""
    B, m = len(lens), max(max(lens), 1)
    max_len = m if max_len is None else max_len
    if page:
        pages, n = table(B, -(-m // page), page, seed)
        kw, of = dict(pages=pages, page_rows=page), lambda b, s: L.row_of(pages.cpu(), page, None, b, s)
    else:
        off = ints(*np.concatenate([[2], 2 + np.cumsum(lens)[:-1]]).tolist())
        n, firsts = 5 + sum(lens), off.tolist()
        kw, of = dict(off=off), lambda b, s: firsts[b] + s
    rows = cache(C, n, R, rd, seed, spread) if rows is None else rows(n)
    poison(rows, {of(b, s) for b in range(B) for s in range(min(lens[b], max_len))})
    q = torch.randn((B, Lq, H, R + rd), generator=rng(seed + 1)).to(BF16) if q is None else q
    scale = (R + rd) ** -0.5 * 1.7 if scale is None else scale
    pos = ints(*[x - Lq for x in lens])
    lse = torch.full((B, Lq, H), 7.0, device="cuda")
    o = C.latent_attn_decode(q.cuda(), rows, pos, scale, max_len, lse=lse, **kw)
    assert C.csa_device_error() == 0
    lat, rope = L.dequant(rows.fp8, rows.rope, rows.scale)
    ref = L.decode(q, lat, rope, of, pos.tolist(), scale, max_len, rows.scale)
    L.check_attention(o, lse, ref, R + rd, m, V_STEP, f"{lens} H{H} Lq{Lq} R{R} page{page}")
    return o, lse


LENS = [1, 63, 64, 65, 0, 200, 128]


@pytest.mark.parametrize("page", [0, 1, 16, 48, 64, 128])
@pytest.mark.parametrize("H,Lq", [(1, 1), (16, 1), (20, 3), (64, 1), (128, 1), (128, 2)])
def test_decode(C, page, H, Lq):
    run_decode(C, LENS if H * Lq < 128 else LENS[:4], H, Lq, 512, 64, page, seed=H + Lq)
    assert C.csa_last_path() == C.CSA_PATH_LATENT_DECODE_TC


@pytest.mark.parametrize("R,rd", [(32, 16), (128, 32), (256, 64), (512, 128), (480, 64)])
@pytest.mark.parametrize("H,Lq", [(3, 1), (40, 2)])
def test_decode_other_shapes(C, R, rd, H, Lq):
    run_decode(C, LENS, H, Lq, R, rd, 16, seed=R)
    assert C.csa_last_path() == C.CSA_PATH_LATENT_DECODE_GENERIC


@pytest.mark.parametrize("lens", [[1], [2], [4096], [3000, 1, 2999, 7], [130] * 9, [1] * 70, [0, 0], [0, 0, 500]])
def test_decode_splits(C, lens):
    """One sequence over many CTAs, many sequences in one CTA, runs that end at a CTA's end."""
    run_decode(C, lens, 8, 1, 512, 64, 64, seed=len(lens))


@pytest.mark.parametrize("lens,H,Lq,R,rd", [
    ([150 + 37 * i for i in range(38)], 128, 1, 512, 64),                 # few parts of many rows: 16 rows at a time
    ([3 * i for i in range(41)] + [900] * 9, 101, 1, 512, 64),            # of which the last are 5
    ([260 + 11 * i for i in range(45)], 107, 1, 160, 32),                 # channels that are no whole groups of 128
    ([20000], 17, 1, 512, 64), ([20000], 3, 3, 96, 16), ([9000], 66, 1, 512, 64),  # many parts: 4 rows at a time, 1 or 2 left
    ([1200, 2500, 1700, 5, 2900], 5, 1, 512, 64), ([300, 2500, 100], 9, 1, 224, 16),
    ([1200] * 12, 7, 1, 512, 64)])                                        # parts between the two
def test_decode_merges(C, lens, H, Lq, R, rd):
    run_decode(C, lens, H, Lq, R, rd, 64, seed=H)


@pytest.mark.parametrize("R", [512, 256])
def test_decode_many_row_blocks(C, R):
    """More row blocks than lie side by side (40 of 32 rows), and some that do, over cut runs."""
    run_decode(C, [700, 10, 300], 128, 10, R, 64, 64)
    run_decode(C, [2000, 10, 900], 16, 5, R, 64, 64)


@pytest.mark.parametrize("Lq", [4, 64])
def test_decode_several_tokens_and_padding(C, Lq):
    """Tokens in front of position 0 see nothing: zeros and -inf (checked inside)."""
    run_decode(C, [0, 1, Lq - 1, Lq, 3 * Lq + 1], 4, Lq, 512, 64, 16)


def test_decode_max_len_cuts(C):
    """Positions from max_len on are not seen, nor read (they hold NaN)."""
    run_decode(C, [100, 64, 3], 16, 2, 512, 64, 16, max_len=64)
    run_decode(C, [100, 64, 3], 16, 2, 256, 64, 16, max_len=64)


@pytest.mark.parametrize("R", [512, 256])
def test_decode_row_scales(C, R):
    """Rows of very different sizes, zero rows, all-equal and one-sided scores."""
    run_decode(C, [300, 65], 16, 1, R, 64, 16, spread=4.0)

    def zeros(n):
        rows = cache(C, n, R, 64, 9)
        rows.fp8[::3] = 0
        rows.scale[::3] = 1.0
        return rows
    run_decode(C, [300, 65], 16, 1, R, 64, 16, rows=zeros)
    run_decode(C, [300, 65], 16, 1, R, 64, 16, scale=0.0)
    run_decode(C, [300, 65], 16, 1, R, 64, 16, scale=1.0)   # scores of +-100: one key takes all
    run_decode(C, [300, 65], 16, 1, R, 64, 16, scale=-0.05)


def test_decode_a_far_sink_keeps_the_rest(C):
    """A key that outweighs every other by e^12 at 4,000 positions: the others' share is held to the same
    relative error of what they add up to as any."""
    R, n = 512, 4000
    q = torch.randn((1, 1, 16, R + 64), generator=rng(3)).to(BF16)
    q[..., R:] = 0
    q[..., R] = 1.0

    def rows(k):
        r = cache(C, k, R, 64, 4)
        r.rope[:, 0] = 0
        r.rope[2, 0] = 12.0
        r.fp8[2] = 0
        return r
    o, lse = run_decode(C, [n], 16, 1, R, 64, 0, q=q, rows=rows, scale=1.0 / 64)
    run_decode(C, [n], 16, 1, R, 64, 0, q=(q * 64).to(BF16), rows=rows, scale=1.0 / 64)


@pytest.mark.parametrize("size", [2.0 ** -40, 1.0, 2.0 ** 30])
def test_decode_query_sizes(C, size):
    """Queries whose bf16 values lie outside fp16's range (the scale makes up for it)."""
    q = (torch.randn((2, 1, 16, 576), generator=rng(8)) * size).to(BF16)
    q[:, :, 3] = 0
    run_decode(C, [77, 130], 16, 1, 512, 64, 16, q=q, scale=0.07 / size)


@pytest.mark.parametrize("R", [512, 256])
def test_decode_refused_pages_are_skipped(C, R):
    """A missing page's keys are left out of the sums, and reported."""
    H, page = 16, 16
    rows = cache(C, 8 * page, R, 64, 5)
    pages = torch.tensor([[1, 99, 3], [4, -1, 6]], dtype=I32, device="cuda")
    q = torch.randn((2, 1, H, R + 64), generator=rng(2)).to(BF16)
    pos = ints(60, 40)  # the first sequence ends behind the table
    lse = torch.empty((2, 1, H), device="cuda")
    o = C.latent_attn_decode(q.cuda(), rows, pos, 0.05, 64, pages=pages, page_rows=page, lse=lse)
    assert C.csa_device_error() == C.CSA_DEVERR_INDEX
    lat, rope = L.dequant(rows.fp8, rows.rope, rows.scale)
    ref = L.decode(q, lat, rope, lambda b, s: L.row_of(pages.cpu(), page, None, b, s), pos.tolist(), 0.05, 64, rows.scale)
    L.check_attention(o, lse, ref, R + 64, 64, V_STEP)


def test_decode_runs_that_begin_or_end_outside_the_cache(C):
    """Contiguous rows of which the first or the last lie outside are left out of the sums, and reported."""
    rows = cache(C, 300, 512, 64)
    q = torch.randn((3, 1, 8, 576), generator=rng(2)).to(BF16)
    pos, off = ints(150, 200, 20), ints(-5, 211, 100000)
    lse = torch.empty((3, 1, 8), device="cuda")
    o = C.latent_attn_decode(q.cuda(), rows, pos, 0.05, 256, off=off, lse=lse)
    assert C.csa_device_error() == C.CSA_DEVERR_INDEX
    lat, rope = L.dequant(rows.fp8, rows.rope, rows.scale)
    ref = L.decode(q, lat, rope, lambda b, s: int(off[b]) + s, pos.tolist(), 0.05, 256, rows.scale)
    L.check_attention(o, lse, ref, 576, 256, V_STEP)


@pytest.mark.parametrize("page", [8, 32, 256, 384])
def test_decode_page_sizes(C, page):
    """The other sizes that boxes are made of, in a cache of whole groups of 8 rows, and one that is not."""
    run_decode(C, [1000, 385, 7], 16, 1, 512, 64, page)

    run_decode(C, [100, 385, 7], 16, 1, 512, 64, page, rows=lambda n: cache(C, n + 5, 512, 64, 3))


def test_decode_last_page_ends_behind_the_cache(C):
    """A page of which only some rows are in the cache: the others are left out, and reported."""
    for n in (40 * 8, 40 * 8 - 3):
        rows = cache(C, n, 512, 64, 5)
        pages = torch.tensor([[2, 0], [1, 2]], dtype=I32, device="cuda")  # pages of 128 rows; the third has 64 or 61
        q = torch.randn((2, 1, 8, 576), generator=rng(2)).to(BF16)
        pos = ints(255, 255)
        lse = torch.empty((2, 1, 8), device="cuda")
        o = C.latent_attn_decode(q.cuda(), rows, pos, 0.05, 256, pages=pages, page_rows=128, lse=lse)
        assert C.csa_device_error() == C.CSA_DEVERR_INDEX
        lat, rope = L.dequant(rows.fp8, rows.rope, rows.scale)
        ref = L.decode(q, lat, rope, lambda b, s: L.row_of(pages.cpu(), 128, None, b, s), pos.tolist(), 0.05, 256, rows.scale)
        L.check_attention(o, lse, ref, 576, 256, V_STEP)


def test_decode_positions_out_of_any_range(C):
    rows = cache(C, 64, 512, 64)
    q = torch.randn((3, 2, 8, 576), generator=rng(2)).to(BF16)
    pos = ints(-2 ** 63, 2 ** 63 - 1, 5)
    o = C.latent_attn_decode(q.cuda(), rows, pos, 0.05, 20, off=ints(0, 20, 40))
    assert C.csa_device_error() == 0
    lat, rope = L.dequant(rows.fp8, rows.rope, rows.scale)
    ref = L.decode(q, lat, rope, lambda b, s: 20 * b + s, [-100, 100, 5], 0.05, 20, rows.scale)
    L.check_attention(o, None, ref, 576, 20, V_STEP)


def test_decode_rows_behind_four_gigabytes(C):
    """A cache whose last rows lie past 2^32 bytes (and 2^31 elements)."""
    n = (1 << 32) // 512 + 4096
    rows = C.KvRows.empty(n, 576, 64, "cuda")
    tail = cache(C, 4096, 512, 64, 6)
    for a, b in zip((rows.fp8, rows.rope, rows.scale), (tail.fp8, tail.rope, tail.scale)):
        a[n - 4096:] = b
    q = torch.randn((2, 1, 16, 576), generator=rng(2)).to(BF16).cuda()
    pos = ints(300, 700)
    far, near = ints(n - 4096, n - 2048), ints(0, 2048)
    assert torch.equal(C.latent_attn_decode(q, rows, pos, 0.05, 1024, off=far), C.latent_attn_decode(q, tail, pos, 0.05, 1024, off=near))
    a, b = C.latent_gather(rows, ints(0, 5, 11), n=11, off=far), C.latent_gather(tail, ints(0, 5, 11), n=11, off=near)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x = torch.randn((2, 576), generator=rng(1)).cuda()
    C.latent_append(x, ints(9, 10), rows, off=far)
    C.latent_append(x, ints(9, 10), tail, off=near)
    assert torch.equal(rows.fp8[n - 4096:], tail.fp8) and C.csa_device_error() == 0


# ------------------------------------------------------------------------------------------
# prefill
# ------------------------------------------------------------------------------------------

def run_prefill(C, nq, nk, H, dims, dtype, causal, seed=0, scale=None, gap=3, size=1.0, k_rope_bias=0.0):
    """Packed sequences with `gap` rows of NaN behind the last, against the formula."""
    dn, dr, dv = dims
    cq, ck = np.concatenate([[0], np.cumsum(nq)]), np.concatenate([[0], np.cumsum(nk)])
    g = rng(seed)
    q = torch.randn((cq[-1] + gap, H, dn + dr), generator=g)
    kv = torch.randn((ck[-1] + gap, H, dn + dv), generator=g) * size
    kr = torch.randn((ck[-1] + gap, dr), generator=g) + k_rope_bias
    q, kv, kr = (t.to(dtype) for t in (q, kv, kr))
    if gap:
        q[cq[-1]:], kv[ck[-1]:], kr[ck[-1]:] = (float("nan"),) * 3
    scale = (dn + dr) ** -0.5 * 1.7 if scale is None else scale
    o = torch.full((len(q), H, dv), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((len(q), H), 7.0, device="cuda")
    C.latent_attn_prefill(q.cuda(), kv.cuda(), kr.cuda(), ints(*cq), ints(*ck), max(max(nq), 1), scale, causal, o=o, lse=lse)
    assert C.csa_device_error() == 0
    n = int(cq[-1])
    ref = [t[:n] for t in L.prefill(q, kv, kr, cq.tolist(), ck.tolist(), dn, scale, causal)]
    L.check_attention(o[:n], lse[:n], ref, dn + dr, max(max(nk), 1), L.STEP[dtype], f"{nq} {nk} H{H} {dims} {dtype} causal={causal}")
    assert (o[n:] == 7).all() and (lse[n:] == 7).all()  # rows behind the last sequence
    return o, lse


SPLIT = [([1], [1100], 1), ([256], [5000], 4), ([100, 300], [2500, 900], 2), ([5, 0, 40], [4000, 700, 0], 3), ([130], [20000], 1),
         ([33, 7], [1, 9000], 2), ([1300], [4100], 30), ([700, 1, 300], [3900, 4000, 8000], 18)]  # the last two: full rounds, then parts


@pytest.mark.parametrize("nq,nk,H", SPLIT)
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_few_queries_many_keys(C, nq, nk, H, causal):
    """Keys split over the SMs: a row's parts merged, parts with nothing to see, sequences shorter than the parts."""
    n = [sum(x) + 3 for x in (nq, nk)]
    assert C.latent_attn_prefill_workspace_size(len(nq), *n, H, 128, 64, 128, max(nq)) > 0
    run_prefill(C, nq, nk, H, (128, 64, 128), BF16, causal, seed=H, size=3.0)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 20.0])
def test_prefill_split_scales(C, scale):
    run_prefill(C, [70], [2000], 2, (128, 64, 128), BF16, True, scale=scale)


def test_prefill_split_or_not(C):
    """With and without a workspace the sums differ in their order alone; a workspace that is too small is refused; what is
    not finite in a part reaches its rows."""
    g = rng(3)
    q, kv, kr = (torch.randn(s, generator=g).to(BF16).cuda() for s in ((40, 2, 192), (4000, 2, 256), (4000, 64)))
    cq, ck = ints(0, 40), ints(0, 4000)
    size = C.latent_attn_prefill_workspace_size(1, 40, 4000, 2, 128, 64, 128, 40)
    o, whole = torch.empty((2, 40, 2, 128), dtype=BF16, device="cuda")
    lse, whole_lse = torch.empty((2, 40, 2), device="cuda")
    ws = torch.empty((size,), dtype=torch.uint8, device="cuda")
    C.latent_attn_prefill(q, kv, kr, cq, ck, 40, 0.1, o=o, lse=lse, workspace=ws)
    args = [t.data_ptr() for t in (q, kv, kr, cq, ck)] + [1, 40, 4000, 2, 128, 64, 128, 40, 0.1, 1, C.CSA_BF16]
    st = torch.cuda.current_stream().cuda_stream
    assert C.lib().latent_attn_prefill(*args, whole.data_ptr(), whole_lse.data_ptr(), None, 0, st) == C.CSA_OK
    # each is off the formula's result by a rounding of P and of o: two bf16 steps of either, of values below 4
    assert (o.float() - whole.float()).abs().max() <= 4 * 2 ** -8 * whole.float().abs().max()
    # the sums' terms are off by 2^-22 each (the exponential) and 2^-24 a rounding of the sum, lse (about 9) by 2^-21
    assert (lse - whole_lse).abs().max() < 1e-5
    with pytest.raises(C.CsaError):
        C.latent_attn_prefill(q, kv, kr, cq, ck, 40, 0.1, workspace=ws[:size - 1])
    kv[3000, 1, :] = float("nan")
    bad = C.latent_attn_prefill(q, kv, kr, cq, ck, 40, 0.1)
    assert bad[:, 1].isnan().all() and torch.equal(bad[:, 0], o[:, 0])


RAGGED = [([1], [1]), ([128], [128]), ([129, 0, 1, 127], [129, 0, 1, 127]), ([5, 300, 64], [5, 300, 64]),
          ([3, 1, 130, 20], [200, 129, 130, 0]), ([40, 260], [17, 255]), ([0, 0], [4, 0]), ([257], [513])]


@pytest.mark.parametrize("nq,nk", RAGGED)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H", [1, 5])
def test_prefill(C, nq, nk, causal, H):
    run_prefill(C, nq, nk, H, (128, 64, 128), BF16, causal, seed=H)
    if sum(nq):
        assert C.csa_last_path() == C.CSA_PATH_LATENT_PREFILL_TC


@pytest.mark.parametrize("dims,dtype", [((128, 64, 128), F32), ((16, 16, 16), BF16), ((64, 32, 96), F32), ((192, 64, 256), BF16)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_other_shapes(C, dims, dtype, causal):
    for nq, nk in RAGGED:
        run_prefill(C, nq, nk, 3, dims, dtype, causal, seed=dims[0])
    assert C.csa_last_path() == C.CSA_PATH_LATENT_PREFILL_GENERIC


def test_prefill_longer(C):
    run_prefill(C, [700, 33], [1500, 33], 2, (128, 64, 128), BF16, True, seed=4)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.1])
def test_prefill_scores(C, scale):
    """All-equal, one-sided and negated scores."""
    run_prefill(C, [200, 64], [260, 64], 2, (128, 64, 128), BF16, True, scale=scale)


def test_prefill_rising_scores(C):
    """Scores that rise along the keys, so that the running maximum moves in every tile."""
    n, H = 600, 2
    g = rng(3)
    q = torch.randn((n, H, 192), generator=g).to(BF16)
    kv = torch.randn((n, H, 256), generator=g).to(BF16)
    kr = torch.randn((n, 64), generator=g)
    q[..., 128] = 4.0
    kr[:, 0] = torch.arange(n) * 0.25
    kr = kr.to(BF16)
    lse = torch.empty((n, H), device="cuda")
    o = C.latent_attn_prefill(q.cuda(), kv.cuda(), kr.cuda(), ints(0, n), ints(0, n), n, 0.3, lse=lse)
    ref = L.prefill(q, kv, kr, [0, n], [0, n], 128, 0.3, True)
    L.check_attention(o, lse, ref, 192, n, L.STEP[BF16])


def test_prefill_hidden_rows_may_hold_anything(C):
    """NaN and infinities in another sequence's rows do not reach this one's."""
    n = [70, 50, 90]
    cu = np.concatenate([[0], np.cumsum(n)])
    g = rng(7)
    q, kv, kr = (torch.randn(s, generator=g).to(BF16).cuda() for s in ((210, 2, 192), (210, 2, 256), (210, 64)))
    good = C.latent_attn_prefill(q, kv, kr, ints(*cu), ints(*cu), 90, 0.1)
    kv[70:120], kr[70:120] = float("nan"), float("inf")
    o = C.latent_attn_prefill(q, kv, kr, ints(*cu), ints(*cu), 90, 0.1)
    assert torch.equal(o[:70], good[:70]) and torch.equal(o[120:], good[120:])


def test_prefill_max_q_bounds_the_queries(C):
    """Queries past max_q are not computed, the others are as without it."""
    g = rng(9)
    q, kv, kr = (torch.randn(s, generator=g).to(BF16).cuda() for s in ((300, 2, 192), (300, 2, 256), (300, 64)))
    full = C.latent_attn_prefill(q, kv, kr, ints(0, 300), ints(0, 300), 300, 0.1)
    o = torch.full_like(full, 7.0)
    C.latent_attn_prefill(q, kv, kr, ints(0, 300), ints(0, 300), 100, 0.1, o=o)
    assert torch.equal(o[:100], full[:100]) and (o[100:] == 7).all()


# ------------------------------------------------------------------------------------------
# as they are used
# ------------------------------------------------------------------------------------------

class Layer:
    """A latent attention layer's weights and cache, and its two ways to attend."""
    H, R, rd, dn, dv, page = 16, 512, 64, 128, 128, 64

    def __init__(self, C, B, L_max, seed):
        g = rng(seed)
        self.C, self.B = C, B
        self.U = (torch.randn((self.H, self.dn, self.R), generator=g) / self.R ** 0.5).to(BF16).cuda()
        self.W = (torch.randn((self.H, self.dv, self.R), generator=g) / self.R ** 0.5).to(BF16).cuda()
        self.gain = (1 + 0.1 * torch.randn((self.R,), generator=g)).cuda()
        self.pages, n = table(B, -(-L_max // self.page), self.page, seed)
        self.rows = C.KvRows.empty(n, self.R + self.rd, self.rd, "cuda")
        self.scale = (self.dn + self.rd) ** -0.5
        self.L_max = L_max

    def append(self, x, seq, pos):
        self.C.latent_append(x, pos, self.rows, g=self.gain, base=10000.0, seq=seq, pages=self.pages, page_rows=self.page)

    def prefill(self, q, lens, nq):
        """The last nq[b] of lens[b] tokens attend, expanded from what the cache holds."""
        cq, ck = (ints(*np.concatenate([[0], np.cumsum(v)]).tolist()) for v in (nq, lens))
        lat, rope = self.C.latent_gather(self.rows, ck, n=sum(lens), pages=self.pages, page_rows=self.page)
        kv = torch.einsum("nr,hdr->nhd", lat, torch.cat([self.U, self.W], 1)).contiguous()
        return self.C.latent_attn_prefill(q, kv, rope, cq, ck, max(nq), self.scale)

    def decode(self, q, pos):
        """q [B, Lq, H, dn + rd]: absorbed, and out of the latent space again."""
        qa = torch.cat([torch.einsum("bjhd,hdr->bjhr", q[..., :self.dn], self.U), q[..., self.dn:]], -1)
        o = self.C.latent_attn_decode(qa, self.rows, pos, self.scale, self.L_max, pages=self.pages, page_rows=self.page)
        return torch.einsum("bjhr,hdr->bjhd", o, self.W)


def test_a_layer_prompts_then_decodes(C):
    """Prompts in two chunks, then decode steps of one and of three tokens: a token's output in the absorbed
    form is its output in the expanded one.  The two forms round to bf16 at different places -- the
    absorbed query, the expanded key and value, the two outputs: at most six roundings of 2^-8 on terms
    that add up like random signs (sqrt of 192 and more terms), so a row is within 4 half steps of its
    largest value."""
    B, lens = 3, [90, 200, 131]
    lay = Layer(C, B, 320, 1)
    g = rng(2)
    new = [1, 1, 3]
    total = [n + sum(new) for n in lens]
    x = [torch.randn((t, 576), generator=g).to(BF16).cuda() for t in total]
    q = [torch.randn((t, lay.H, 192), generator=g).to(BF16).cuda() for t in total]

    def rows(a, b):  # the tokens a[i] .. b[i] - 1 of every sequence, packed
        seq = torch.cat([torch.full((b[i] - a[i],), i, dtype=I32) for i in range(B)]).cuda()
        pos = torch.cat([torch.arange(a[i], b[i]) for i in range(B)]).cuda()
        return torch.cat([x[i][a[i]:b[i]] for i in range(B)]), torch.cat([q[i][a[i]:b[i]] for i in range(B)]), seq, pos
    half = [40, 200, 64]
    for a, b in (([0] * 3, half), (half, lens)):
        xs, qs, seq, pos = rows(a, b)
        if len(xs):
            lay.append(xs, seq, pos)
            out = lay.prefill(qs, list(b), [v - u for u, v in zip(a, b)])
    at = list(lens)
    got = []
    for n in new:
        xs, qs, seq, pos = rows(at, [v + n for v in at])
        lay.append(xs, seq, pos)
        got.append(lay.decode(qs.view(B, n, lay.H, 192), ints(*at)))
        at = [v + n for v in at]
    assert C.csa_device_error() == 0
    # every new token again, in the expanded form
    out = lay.prefill(torch.cat([q[i][lens[i]:] for i in range(B)]), total, [sum(new)] * B).view(B, sum(new), lay.H, 128)
    got = torch.cat(got, 1)
    err = (got.float() - out.float()).abs().amax(-1) / out.float().abs().amax(-1)
    assert err.max() <= 4 * 2.0 ** -8, float(err.max())


def test_captured_and_replayed_on_other_streams(C):
    """A decode step (append and attention) captured once and replayed with new tokens, beside another
    graph with a workspace of its own, gives what the plain calls give."""
    lay = [Layer(C, 4, 256, s) for s in (3, 4)]
    g = rng(5)
    seq = torch.arange(4, dtype=I32, device="cuda")
    state = []
    for la in lay:
        for t in (la.rows.fp8, la.rows.rope, la.rows.scale):
            t.zero_()
        x0 = torch.randn((4 * 100, 576), generator=g).to(BF16).cuda()
        la.append(x0, seq.repeat_interleave(100), torch.arange(100, device="cuda").repeat(4))
        st = dict(x=torch.empty((4, 576), dtype=BF16, device="cuda"), pos=torch.empty((4,), dtype=I64, device="cuda"),
                  q=torch.empty((4, 1, 16, 576), dtype=BF16, device="cuda"), o=torch.empty((4, 1, 16, 512), dtype=BF16, device="cuda"),
                  ws=torch.empty((C.latent_attn_decode_workspace_size(4, 1, 16, 512, 256),), dtype=torch.uint8, device="cuda"))
        st["x"].zero_(), st["pos"].fill_(100), st["q"].zero_()
        state.append(st)

    def step(la, st, o, rows):
        C.latent_append(st["x"], st["pos"], rows, g=la.gain, base=10000.0, seq=seq, pages=la.pages, page_rows=la.page)
        C.latent_attn_decode(st["q"], rows, st["pos"], la.scale, 256, pages=la.pages, page_rows=la.page, o=o, workspace=st["ws"])
    graphs = []
    for la, st in zip(lay, state):
        step(la, st, st["o"], la.rows)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(la, st, st["o"], la.rows)
        graphs.append(gr)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for t in range(3):
        want = []
        for la, st in zip(lay, state):
            st["x"].copy_(torch.randn((4, 576), generator=g))
            st["q"].copy_(torch.randn((4, 1, 16, 576), generator=g))
            st["pos"].copy_(torch.tensor([100 + t, 100, 101 + 2 * t, 150]))
            o = torch.empty_like(st["o"])
            rows = C.KvRows(la.rows.fp8.clone(), la.rows.rope.clone(), la.rows.scale.clone())
            step(la, st, o, rows)
            want.append((o, rows))
        torch.cuda.synchronize()
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for la, st, (o, rows) in zip(lay, state, want):
            assert torch.equal(st["o"], o) and torch.equal(la.rows.fp8, rows.fp8) and torch.equal(la.rows.rope, rows.rope)
    assert C.csa_device_error() == 0


def test_the_same_call_gives_the_same_bits(C):
    rows = cache(C, 4096, 512, 64)
    q = torch.randn((4, 1, 64, 576), generator=rng(1)).to(BF16).cuda()
    pos, off = ints(900, 3, 1023, 500), ints(0, 1024, 2048, 3000)
    a = C.latent_attn_decode(q, rows, pos, 0.05, 1024, off=off)
    qp, kv, kr = (torch.randn(s, generator=rng(2)).to(BF16).cuda() for s in ((700, 4, 192), (700, 4, 256), (700, 64)))
    p = C.latent_attn_prefill(qp, kv, kr, ints(0, 700), ints(0, 700), 700, 0.1)
    for _ in range(5):
        assert torch.equal(a, C.latent_attn_decode(q, rows, pos, 0.05, 1024, off=off))
        assert torch.equal(p, C.latent_attn_prefill(qp, kv, kr, ints(0, 700), ints(0, 700), 700, 0.1))


def test_a_side_stream_is_used(C):
    """The call goes to the stream that is current, or to the one that is named."""
    rows = cache(C, 2048, 512, 64)
    q = torch.randn((2, 1, 16, 576), generator=rng(1)).to(BF16).cuda()
    pos, off = ints(900, 800), ints(0, 1024)
    ref = C.latent_attn_decode(q, rows, pos, 0.05, 1024, off=off)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    late = torch.zeros_like(q)
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late.copy_(q)
        a = C.latent_attn_decode(late, rows, pos, 0.05, 1024, off=off)
    ws = torch.empty((C.latent_attn_decode_workspace_size(2, 1, 16, 512, 1024),), dtype=torch.uint8, device="cuda")
    b = torch.empty_like(ref)
    C.latent_attn_decode(late, rows, pos, 0.05, 1024, off=off, o=b, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(a, ref) and torch.equal(b, ref)


@pytest.mark.parametrize("as_handle", [False, True])
def test_what_a_call_allocates_belongs_to_its_stream(C, as_handle):
    """Workspaces and outputs of a call on a named stream are not given to the current stream's tensors while it runs."""
    rows = cache(C, 4096, 512, 64)
    q = torch.randn((1, 1, 16, 576), generator=rng(1)).to(BF16).cuda()
    pos, off = ints(4000), ints(0)
    qp, kv, kr = (torch.randn(s, generator=rng(2)).to(BF16).cuda() for s in ((8, 2, 192), (4000, 2, 256), (4000, 64)))
    cu, cq, ck = ints(0, 4000), ints(0, 8), ints(0, 4000)

    def calls(stream):
        return (C.latent_attn_decode(q, rows, pos, 0.05, 4096, off=off, stream=stream),
                C.latent_attn_prefill(qp, kv, kr, cq, ck, 8, 0.1, stream=stream), *C.latent_gather(rows, cu, n=4000, off=off, stream=stream))
    ref = calls(None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
    got = calls(s.cuda_stream if as_handle else s)
    n = [C.latent_attn_decode_workspace_size(1, 1, 16, 512, 4096), C.latent_attn_prefill_workspace_size(1, 8, 4000, 2, 128, 64, 128, 8)]
    over = [torch.full((k,), 255, dtype=torch.uint8, device="cuda") for k in n for _ in range(3)]  # would be NaN in the workspaces
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref)) and len(over) == 6
    bare = calls(0)  # the default stream, by its handle
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bare, ref))
