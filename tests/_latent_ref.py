"""The latent attention operators in 64 bits on the CPU, straight from their formulas, and the error
bounds that their kernels are held to (not collected by pytest)."""
import torch

F64 = torch.float64
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step of a rounding, relative


def row_of(pages, page_rows, off, b, s):
    """Cache row of position s of sequence b, or None when the page table ends before it."""
    if pages is None:
        return int(off[b]) + s
    if s // page_rows >= pages.shape[1]:
        return None
    return int(pages[b, s // page_rows]) * page_rows + s % page_rows


def dequant(fp8, rope, scale):
    """(lat, rope) of cache rows in 64 bits."""
    return fp8.cpu().view(torch.float8_e4m3fn).to(F64) * scale.cpu().to(F64)[:, None], rope.cpu().to(F64)


def append_rows(x, pos, R, g=None, eps=1e-6, base=0.0):
    """(lat [n, R], rope [n, rd]) before they are quantised."""
    x = x.cpu().to(F64)
    u, v = x[:, :R], x[:, R:]
    if g is not None:
        u = u / torch.sqrt((u * u).mean(1, keepdim=True) + eps) * g.cpu().to(F64)
    if base:
        rd = v.shape[1]
        k = torch.arange(rd // 2, dtype=F64)
        a = pos.cpu().to(F64)[:, None] * base ** (-2 * k / rd)
        e, o = v[:, 0::2], v[:, 1::2]
        v = torch.stack([e * a.cos() - o * a.sin(), e * a.sin() + o * a.cos()], -1).flatten(1)
    return u, v


def attend(q, k, v, seen, scale, v_scale=None):
    """One head: q [n, d], k [m, d], v [m, e], seen [n, m].  Returns o, lse, and what the error bound
    needs: sum p|v| / sum p, the largest scale * sum |q||k| of a seen key and, with the values' row
    scales, the largest p v_scale of a seen key times sum |v| / v_scale."""
    o = torch.zeros((len(q), v.shape[1]), dtype=F64)
    lse = torch.full((len(q),), -torch.inf, dtype=F64)
    size = torch.zeros_like(o)
    mag = torch.zeros_like(lse)
    small = torch.zeros_like(o)
    for i in range(len(q)):
        at = seen[i].nonzero()[:, 0]
        if not len(at):
            continue
        z = (k[at] @ q[i]) * scale
        lse[i] = torch.logsumexp(z, 0)
        p = torch.exp(z - lse[i])
        o[i], size[i] = p @ v[at], p @ v[at].abs()
        mag[i] = (k[at].abs() @ q[i].abs()).max() * abs(scale)
        if v_scale is not None:
            small[i] = (p * v_scale[at]).max() * (v[at].abs() / v_scale[at][:, None]).sum(0)
    return o, lse, size, mag, small


def check_attention(o, lse, ref, dk, n_keys, p_step, name=""):
    """Kernel outputs against attend()'s.  A score is a sum of dk products in fp32 (off by at most dk
    half steps of the sum of their magnitudes, and 8 more for the scale and log2 e), so a probability
    is off by twice that relative; its own rounding to p_step and the fp32 sum over n_keys come on top,
    and the output's rounding at the end.  `small` is not zero where the probabilities times the row
    scales, w, are held as 8-bit floats in two terms: with M their largest, the unit that they are
    held in is at most 2^-2.5 M (it is set so that the largest becomes 2^2.5 to 2^3.5, and only a larger one,
    or one that would matter beside the sum, sets it again), and below 2^-6 units, where the first term is
    off by up to 2^-10, the second has 3 bits of that left: they are off by up to 2^-13 units, so each by
    at most 2^-15.5 M beyond p_step."""
    ro, rl, size, mag, small = ref
    dz = (dk + 8) * 2.0 ** -24 * mag
    tau = 2 * dz + p_step + (n_keys + 8) * 2.0 ** -24 + 2.0 ** -20
    tol = STEP[o.dtype] * ro.abs() + (tau[..., None] * size + 2.0 ** -15.5 * small) * 1.01 + 1e-30
    got = o.cpu().to(F64)
    assert torch.isfinite(got).all(), name
    bad = (got - ro).abs() > tol
    assert not bad.any(), (name, bad.nonzero()[:4].tolist(), float(((got - ro).abs() / tol).max()))
    if lse is not None:
        got = lse.cpu().to(F64)
        none = torch.isinf(rl)
        assert torch.equal(none, torch.isinf(got)) and (got[none] < 0).all(), name
        err = (got - rl).abs()[~none]
        # the sum of unrounded probabilities: their error, and the logarithm's
        lim = (2 * dz + (n_keys + 8) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * rl.abs())[~none]
        assert (err <= lim).all(), (name, float((err / lim).max()))


def decode(q, lat, rope, rows_of, pos, scale, max_len, v_scale=None):
    """attend() over every (sequence, token, head): rows_of(b, s) is the cache row or None."""
    B, Lq, H, c = q.shape
    key = torch.cat([lat, rope], 1)
    q = q.cpu().to(F64)
    out = []
    for b in range(B):
        n = max(0, min(int(pos[b]) + Lq, max_len))
        at = [rows_of(b, s) for s in range(n)]
        ok = torch.tensor([r is not None and 0 <= r < len(key) for r in at], dtype=torch.bool)
        at = torch.tensor([r if r is not None and 0 <= r < len(key) else 0 for r in at], dtype=torch.long)
        s = torch.arange(n)
        seen = torch.stack([ok & (s <= int(pos[b]) + j) for j in range(Lq)])  # [Lq, n]
        r = attend(q[b].reshape(Lq * H, c), key[at], lat[at], seen[:, None].expand(Lq, H, n).reshape(Lq * H, n), scale,
                   None if v_scale is None else v_scale.cpu().to(F64)[at])
        out.append([t.reshape(Lq, H, *t.shape[1:]) for t in r])
    return [torch.stack(t) for t in zip(*out)]


def prefill(q, kv, k_rope, cu_q, cu_k, dn, scale, causal):
    q, kv, k_rope = (t.cpu().to(F64) for t in (q, kv, k_rope))
    Tq, H, _ = q.shape
    dv = kv.shape[2] - dn
    o, lse = torch.zeros((Tq, H, dv), dtype=F64), torch.full((Tq, H), -torch.inf, dtype=F64)
    size, mag = torch.zeros_like(o), torch.zeros((Tq, H), dtype=F64)
    for a, b, c, d in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        nq, nk = b - a, d - c
        i, j = torch.arange(nq)[:, None], torch.arange(nk)[None, :]
        seen = (j <= i + nk - nq) if causal else torch.ones((nq, nk), dtype=torch.bool)
        for h in range(H):
            key = torch.cat([kv[c:d, h, :dn], k_rope[c:d]], 1)
            o[a:b, h], lse[a:b, h], size[a:b, h], mag[a:b, h], _ = attend(q[a:b, h], key, kv[c:d, h, dn:], seen, scale)
    return o, lse, size, mag, torch.zeros_like(o)
