"""Timed cases of the latent attention operators: a cache row per token that is one shared latent
vector (FP8 with a row scale) and a rotated part (BF16), what writes and reads such a cache, and
the attention over it in its absorbed form (decode) and its expanded form (prefill).

`run(state)` makes one pass in plain torch, or, with `own` set, through the library.
"""
import math

import torch

own = False

R, RD = 512, 64            # latent channels and rotated channels of a cache row
DN, DV = 128, 128          # expanded form: unrotated key channels and value channels of a head
C = R + RD
EPS, BASE = 1e-6, 10000.0


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def listed():
    return [
        # one user's next token after a few thousand: latency alone
        {"name": "decode 1 x 4k, 16 heads", "op": "decode", "B": 1, "H": 16, "Lq": 1, "L": 4096, "low": 4096, "page": 128},
        # a serving batch of mixed lengths, the heads split over the GPUs of a node
        {"name": "decode 64 mixed, 16 heads", "op": "decode", "B": 64, "H": 16, "Lq": 1, "L": 16384, "low": 1024, "page": 128},
        # the same with every head on each GPU and two tokens of a sequence at once
        {"name": "decode 32 mixed, 128 heads x 2", "op": "decode", "B": 32, "H": 128, "Lq": 2, "L": 12001, "low": 3000, "page": 32},
        # a few very long contexts
        {"name": "decode 4 x 1M, 64 heads", "op": "decode", "B": 4, "H": 64, "Lq": 1, "L": 1048576, "low": 1048576, "page": 128},
        # several short prompts of odd lengths in one batch
        {"name": "prefill 8 short, 16 heads", "op": "prefill", "B": 8, "H": 16, "Lq": 511, "low": 1, "past": 0, "causal": True},
        # one ordinary prompt
        {"name": "prefill 4k, 16 heads", "op": "prefill", "B": 1, "H": 16, "Lq": 4096, "low": 4096, "past": 0, "causal": True},
        # a chunk of two long prompts behind what the cache holds already
        {"name": "prefill 2 x 2k after 14k", "op": "prefill", "B": 2, "H": 16, "Lq": 2048, "low": 1777, "past": 14336, "causal": True},
        # a long prompt in one piece
        {"name": "prefill 16k, 16 heads", "op": "prefill", "B": 1, "H": 16, "Lq": 16384, "low": 16384, "past": 0, "causal": True},
        # a decode step's new rows
        {"name": "append 64 tokens", "op": "append", "B": 64, "n": 1, "L": 4096, "page": 128, "f32": False},
        # a long prompt's rows
        {"name": "append 8 x 8k", "op": "append", "B": 8, "n": 8192, "L": 8192, "page": 128, "f32": False},
        # the held part of a few prompts, for the expanded form of their next chunk
        {"name": "gather 8 x ~1k", "op": "gather", "B": 8, "L": 1500, "low": 333, "page": 32},
        # the same of long ones
        {"name": "gather 8 x ~24k", "op": "gather", "B": 8, "L": 32768, "low": 16384, "page": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "append", "gather"])
    page = rng.choice([16, 32, 64, 128])
    if op == "decode":
        B, H, Lq = _log(rng, 1, 128), rng.choice([8, 16, 20, 32, 64, 96, 128]), rng.choice([1, 1, 1, 2, 3, 4])
        cap = min(2 ** 22 // B, int(2.6e8 / (B * max(H * Lq, 16))))   # keys and scores at most those of the listed cases
        L = max(1, _log(rng, 64, max(65, min(1048576, cap))))
        return {"op": op, "B": B, "H": H, "Lq": min(Lq, L), "L": L, "low": max(min(Lq, L), _log(rng, max(1, L // 16), L)), "page": page}
    if op == "prefill":
        H, B = rng.choice([4, 8, 16, 20, 32, 64]), _log(rng, 1, 16)
        past, causal = rng.choice([0, 0, _log(rng, 64, 32768)]), rng.random() < 0.8
        area = (2.6e8 if causal and not past else 1.3e8) * 16 / (H * B)   # a head's scores: at most those of the listed cases
        Lq = min(16384, _log(rng, 16, max(17, int(area ** 0.5 / 1.01))))
        past = max(0, min(past, int(area) // Lq - Lq))
        return {"op": op, "B": B, "H": H, "Lq": Lq, "low": max(1, _log(rng, max(1, Lq // 8), Lq)), "past": past, "causal": causal}
    if op == "append":
        B = _log(rng, 1, 128)
        n = rng.choice([1, _log(rng, 1, max(2, 65536 // B))])
        return {"op": op, "B": B, "n": n, "L": n + _log(rng, 16, max(17, 131072 // B)), "page": page, "f32": rng.random() < 0.25}
    B = _log(rng, 1, 64)
    L = _log(rng, 16, 262144 // B)
    return {"op": op, "B": B, "L": L, "low": max(1, _log(rng, max(1, L // 8), L)), "page": page}


def _lengths(case, hi, low):
    """Lengths of the case's sequences: the same for every seed, from `low` to `hi`, the longest first."""
    B = case["B"]
    if B == 1:
        return [hi]
    return [max(1, int(round(hi * (low / hi) ** (b / (B - 1))))) for b in range(B)]


def _keys(case):
    lens = _lengths(case, case["L"], case["low"])
    return lens, sum(lens)


def work(case):
    if case["op"] == "decode":
        lens, keys = _keys(case)
        B, H, Lq = case["B"], case["H"], case["Lq"]
        pairs = sum(max(0, n - (Lq - 1 - j)) for n in lens for j in range(Lq))
        return {"bytes": keys * (R + 2 * RD + 4) + B * Lq * H * (2 * C + 2 * R + 4), "flops": 2.0 * H * (C + R) * pairs}
    if case["op"] == "prefill":
        lens, H = _lengths(case, case["Lq"], case["low"]), case["H"]
        pairs = sum(n * (n + 1) // 2 + n * case["past"] if case["causal"] else n * (n + case["past"]) for n in lens)
        q, k = sum(lens), sum(lens) + case["B"] * case["past"]
        return {"bytes": q * H * (2 * (DN + RD) + 2 * DV + 4) + k * (H * 2 * (DN + DV) + 2 * RD), "flops": 2.0 * H * (DN + RD + DV) * pairs}
    if case["op"] == "append":
        n = case["B"] * case["n"]
        return {"bytes": n * (C * (4 if case["f32"] else 2) + R + 2 * RD + 4 + 8), "flops": 8.0 * n * C}
    _, rows = _keys(case)
    return {"bytes": rows * (R + 2 * RD + 4 + 2 * C), "flops": 1.0 * rows * R}


# ------------------------------------------------------------------------------------------
# what a program has in hand
# ------------------------------------------------------------------------------------------

def _cache(g, rows):
    """A cache of rows ~ N(0, 1) in its stored form."""
    fp8 = torch.empty((rows, R), dtype=torch.uint8, device="cuda")
    scale = torch.empty((rows,), dtype=torch.float32, device="cuda")
    rope = torch.empty((rows, RD), dtype=torch.bfloat16, device="cuda")
    for r in range(0, rows, 1 << 19):
        x = torch.randn((min(1 << 19, rows - r), R), generator=g, device="cuda")
        s = x.abs().amax(1) / 448.0
        fp8[r:r + len(x)] = (x / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[r:r + len(x)] = s
        rope[r:r + len(x)] = torch.randn((len(x), RD), generator=g, device="cuda").to(torch.bfloat16)
    return fp8, rope, scale


def _pages(g, case, L):
    """A page table over shuffled pages, and the rows of the cache behind it."""
    per = -(-L // case["page"])
    n = case["B"] * per
    return torch.randperm(n, generator=g, device="cuda").to(torch.int32).view(case["B"], per), n * case["page"]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(case)
    dev = "cuda"
    if case["op"] == "prefill":
        lens, H = _lengths(case, case["Lq"], case["low"]), case["H"]
        cq = [0]
        ck = [0]
        for n in lens:
            cq.append(cq[-1] + n)
            ck.append(ck[-1] + n + case["past"])
        st["q"] = torch.randn((cq[-1], H, DN + RD), generator=g, device=dev).to(torch.bfloat16)
        st["kv"] = torch.randn((ck[-1], H, DN + DV), generator=g, device=dev).to(torch.bfloat16)
        st["k_rope"] = torch.randn((ck[-1], RD), generator=g, device=dev).to(torch.bfloat16)
        st["cu_q"], st["cu_k"] = (torch.tensor(v, dtype=torch.int64, device=dev) for v in (cq, ck))
        st["scale"] = (DN + RD) ** -0.5
        return st
    pages, rows = _pages(g, case, case["L"])
    st["pages"] = pages
    st["fp8"], st["rope"], st["scale_rows"] = _cache(g, rows)
    if case["op"] == "append":
        B, n = case["B"], case["n"]
        x = torch.randn((B * n, C), generator=g, device=dev) * torch.exp(0.5 * torch.randn((B * n, 1), generator=g, device=dev))
        st["x"] = x if case["f32"] else x.to(torch.bfloat16)
        st["gain"] = 1 + 0.1 * torch.randn((R,), generator=g, device=dev)
        first = torch.randint(0, case["L"] - n + 1, (B, 1), generator=g, device=dev)
        st["pos"] = (first + torch.arange(n, device=dev)[None, :]).reshape(-1)
        st["seq"] = torch.arange(B, device=dev, dtype=torch.int32).repeat_interleave(n)
        return st
    lens, keys = _keys(case)
    if case["op"] == "gather":
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        st["cu"], st["rows"] = torch.tensor(cu, dtype=torch.int64, device=dev), cu[-1]
        return st
    B, H, Lq = case["B"], case["H"], case["Lq"]
    st["q"] = torch.randn((B, Lq, H, C), generator=g, device=dev).to(torch.bfloat16)
    st["pos"] = torch.tensor([n - Lq for n in lens], dtype=torch.int64, device=dev)
    st["scale"] = (DN + RD) ** -0.5
    return st


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------

def _rows_of(st, b, s):
    """Cache rows of positions s of sequences b."""
    return st["pages"].long()[b, s // st["page"]] * st["page"] + s % st["page"]


def _softmax(s, seen, v):
    """Softmax over the last axis of the scores s where `seen`, times v; and its log-sum-exp."""
    s = torch.where(seen, s, float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = torch.exp(s - m)
    del s
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(z > 0, z, 1.0)
    return o, (torch.log(z) + m)[..., 0]


def _plain_decode(st):
    B, Lq, H, _ = st["q"].shape
    s = torch.arange(st["L"], device="cuda")
    row = _rows_of(st, torch.arange(B, device="cuda")[:, None], s[None, :].expand(B, -1))
    k = torch.empty((B, st["L"], C), dtype=torch.float32, device="cuda")
    torch.mul(st["fp8"][row].view(torch.float8_e4m3fn).float(), st["scale_rows"][row][..., None], out=k[..., :R])
    k[..., R:] = st["rope"][row].float()
    seen = s[None, None, :] <= (st["pos"][:, None] + torch.arange(Lq, device="cuda")[None, :])[..., None]  # [B, Lq, L]
    z = torch.matmul(st["q"].float().view(B, Lq * H, C), k.transpose(1, 2)) * st["scale"]
    seen = seen[:, :, None, :].expand(B, Lq, H, st["L"]).reshape(B, Lq * H, st["L"])
    o, lse = _softmax(z, seen, k[..., :R])
    return o.view(B, Lq, H, R).to(torch.bfloat16), lse.view(B, Lq, H)


def _plain_prefill(st):
    q, kv, cu_q, cu_k = st["q"], st["kv"], st["cu_q"], st["cu_k"]
    B, H, Lk = len(cu_q) - 1, q.shape[1], st["Lq"] + st["past"]
    i, j = torch.arange(st["Lq"], device="cuda"), torch.arange(Lk, device="cuda")
    nq, nk = (cu_q[1:] - cu_q[:-1])[:, None], (cu_k[1:] - cu_k[:-1])[:, None]
    iq = (cu_q[:-1, None] + i[None, :]).clamp(max=len(q) - 1)
    ik = (cu_k[:-1, None] + j[None, :]).clamp(max=len(kv) - 1)
    k = torch.cat([kv[ik][..., :DN].float(), st["k_rope"][ik].float()[:, :, None, :].expand(-1, -1, H, -1)], -1)
    seen = (j[None, None, :] < nk[:, :, None]) & (i[None, :, None] < nq[:, :, None])
    if st["causal"]:
        seen = seen & (j[None, None, :] <= i[None, :, None] + (nk - nq)[:, :, None])
    z = torch.matmul(q[iq].float().transpose(1, 2), k.permute(0, 2, 3, 1)) * st["scale"]  # [B, H, Lq, Lk]
    o, lse = _softmax(z, seen[:, None], kv[ik][..., DN:].float().transpose(1, 2))
    at = i[None, :] < nq
    return o.transpose(1, 2)[at].to(torch.bfloat16), lse.transpose(1, 2)[at]


def _plain_append(st):
    x = st["x"].double()
    lat = x[:, :R] / torch.sqrt((x[:, :R] ** 2).mean(1, keepdim=True) + EPS) * st["gain"].double()
    lat = lat.float()
    i = torch.arange(RD // 2, device="cuda", dtype=torch.float64)
    a = st["pos"].double()[:, None] * BASE ** (-2.0 * i / RD)[None, :]
    u, v = x[:, R::2], x[:, R + 1::2]
    rot = torch.stack([u * torch.cos(a) - v * torch.sin(a), u * torch.sin(a) + v * torch.cos(a)], -1).flatten(1)
    s = lat.abs().amax(1) / 448.0
    s = torch.where(s > 0, s, 1.0)
    row = _rows_of(st, st["seq"].long(), st["pos"])
    st["fp8"][row] = (lat / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    st["scale_rows"][row] = s
    st["rope"][row] = rot.float().to(torch.bfloat16)
    return st["fp8"].view(torch.float8_e4m3fn), st["rope"], st["scale_rows"]


def _plain_gather(st):
    n = torch.arange(st["rows"], device="cuda")
    b = torch.searchsorted(st["cu"], n, right=True) - 1
    row = _rows_of(st, b, n - st["cu"][b])
    lat = st["fp8"][row].view(torch.float8_e4m3fn).float() * st["scale_rows"][row][:, None]
    return lat.to(torch.bfloat16), st["rope"][row]


def run(st):
    if not own:
        return {"decode": _plain_decode, "prefill": _plain_prefill, "append": _plain_append, "gather": _plain_gather}[st["op"]](st)
    import compressed_sparse_kv_csa_b200 as csa
    if st["op"] == "prefill":
        lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device="cuda")
        o = csa.latent_attn_prefill(st["q"], st["kv"], st["k_rope"], st["cu_q"], st["cu_k"], max_q=st["Lq"], scale=st["scale"],
                                    causal=st["causal"], lse=lse)
        return o, lse
    rows = csa.KvRows(st["fp8"], st["rope"], st["scale_rows"])
    if st["op"] == "decode":
        lse = torch.empty(st["q"].shape[:3], dtype=torch.float32, device="cuda")
        o = csa.latent_attn_decode(st["q"], rows, st["pos"], st["scale"], max_len=st["L"], pages=st["pages"], page_rows=st["page"],
                                   lse=lse)
        return o, lse
    if st["op"] == "append":
        csa.latent_append(st["x"], st["pos"], rows, g=st["gain"], eps=EPS, base=BASE, seq=st["seq"], pages=st["pages"],
                          page_rows=st["page"])
        return st["fp8"].view(torch.float8_e4m3fn), st["rope"], st["scale_rows"]
    return csa.latent_gather(rows, st["cu"], n=st["rows"], pages=st["pages"], page_rows=st["page"])


# ------------------------------------------------------------------------------------------
# the definition in 64 bits, one sequence at a time
# ------------------------------------------------------------------------------------------

def _attend(q, k, v, scale, last):
    """q [H, n, d], k [H or 1, m, d], v [H or 1, m, e] in 64 bits; row i sees keys 0..last[i]."""
    out, lse = [], []
    step = max(1, (1 << 28) // max(1, q.shape[1] * k.shape[1]))
    hidden = torch.arange(k.shape[1], device="cuda")[None, :] > last[:, None]
    for h in range(0, q.shape[0], step):
        kk, vv = (t if t.shape[0] == 1 else t[h:h + step] for t in (k, v))
        z = (q[h:h + step] @ kk.mT).mul_(scale).masked_fill_(hidden, -torch.inf)
        top = z.logsumexp(-1, keepdim=True)
        out.append(z.sub_(top).exp_() @ vv)
        lse.append(top[..., 0])
    return torch.cat(out), torch.cat(lse)


def exact(case, seed):
    st = prepare(case, seed)
    page, f64 = case.get("page", 1), torch.float64
    if case["op"] == "prefill":
        os, ls = [], []
        cq, ck = st["cu_q"].tolist(), st["cu_k"].tolist()
        for a, b, c, d in zip(cq, cq[1:], ck, ck[1:]):
            H, kv = case["H"], st["kv"][c:d].to(f64).permute(1, 0, 2)
            k = torch.cat([kv[..., :DN], st["k_rope"][c:d].to(f64).expand(H, -1, -1)], 2)
            last = torch.arange(b - a, device="cuda") + (d - c) - (b - a) if case["causal"] else torch.full((b - a,), d - c, device="cuda")
            o, lse = _attend(st["q"][a:b].to(f64).permute(1, 0, 2), k, kv[..., DN:], st["scale"], last)
            os.append(o.permute(1, 0, 2))
            ls.append(lse.mT)
        return torch.cat(os), torch.cat(ls)
    table = st["pages"].tolist()
    if case["op"] == "append":
        fp8, rope, sc = st["fp8"].view(torch.float8_e4m3fn).to(f64), st["rope"].to(f64), st["scale_rows"].to(f64)
        where = torch.tensor([table[s][p // page] * page + p % page for s, p in zip(st["seq"].tolist(), st["pos"].tolist())], device="cuda")
        lat, tail = st["x"].to(f64).split([R, RD], 1)
        lat = lat * (lat.pow(2).sum(1, keepdim=True) / R + EPS).rsqrt() * st["gain"].to(f64)
        turn = torch.polar(torch.ones((), dtype=f64, device="cuda"),
                           torch.outer(st["pos"].to(f64), torch.exp(torch.arange(0, RD, 2, dtype=f64, device="cuda") * (-math.log(BASE) / RD))))
        rope[where] = torch.view_as_real(torch.view_as_complex(tail.reshape(-1, RD // 2, 2).contiguous()) * turn).flatten(1)
        sc[where] = lat.abs().max(1).values / 448.0
        # a held value is the nearest one of the 8-bit grid: the grid is part of the definition, so the 8-bit output has no value in 64 bits
        return None, rope, sc
    if case["op"] == "gather":
        lat, tail = [], []
        cu = st["cu"].tolist()
        for b, n in enumerate(y - x for x, y in zip(cu, cu[1:])):
            at = (torch.tensor(table[b], device="cuda")[:, None] * page + torch.arange(page, device="cuda")).flatten()[:n]
            lat.append(st["fp8"].view(torch.float8_e4m3fn)[at].to(f64) * st["scale_rows"][at, None].to(f64))
            tail.append(st["rope"][at].to(f64))
        return torch.cat(lat), torch.cat(tail)
    os, ls = [], []
    for b in range(case["B"]):
        n = int(st["pos"][b]) + case["Lq"]
        at = (torch.tensor(table[b], device="cuda")[:, None] * page + torch.arange(page, device="cuda")).flatten()[:n]
        v = st["fp8"].view(torch.float8_e4m3fn)[at].to(f64) * st["scale_rows"][at, None].to(f64)
        k = torch.cat([v, st["rope"][at].to(f64)], 1)
        o, lse = _attend(st["q"][b].to(f64).transpose(0, 1), k[None], v[None], st["scale"], st["pos"][b] + torch.arange(case["Lq"], device="cuda"))
        os.append(o.transpose(0, 1))
        ls.append(lse.mT)
    return torch.stack(os), torch.stack(ls)
