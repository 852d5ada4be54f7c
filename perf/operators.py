"""What is measured of the paged serving operators: block tables and slot
maps built from request lengths, the rotation and paged write of new keys
and values, and the attention of a batch that shares a long prefix.

A batch of B requests shares a prefix of `prefix` tokens whose keys and
values lie in pages of one pool; every request adds its own tokens in pages
of the same pool.  The three operators are one serving step: tables (which
page and slot each new token gets), write (rotate, store), attention.

A case's request lengths are one fixed list, dealt to the requests in an
order that the seed decides, so that a case's work does not depend on the
seed while its inputs do.
"""

import random

import numpy as np
import torch

own = False

D = 128
THETA = 1.0e6


# -- cases ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 16 running requests (the repository's batch): the smallest launch
        dict(name="tables_decode_16", op="tables", B=16, page=16, cached_lo=1, cached_hi=8192, new=1, long=0,
             long_new=0, pad=0, base=1024),
        # a large batch's step in which a quarter of the requests bring prompts of 4000 tokens
        dict(name="tables_prompts_256", op="tables", B=256, page=64, cached_lo=1, cached_hi=6000, new=1, long=64,
             long_new=4000, pad=100, base=8192),
        # the new tokens of a decode step, 32/8 heads, views of one fused projection
        dict(name="write_decode_16", op="write", n=16, Hq=32, Hkv=8, page=16, dtype="bf16", fused=True, pad=0,
             far=32768),
        # a float32 model's odd-sized chunk, 40/8 heads, rows behind the last token
        dict(name="write_chunk_f32", op="write", n=2531, Hq=40, Hkv=8, page=128, dtype="f32", fused=False, pad=29,
             far=1 << 20),
        # a whole prompt at 32/8 heads, views of one fused projection
        dict(name="write_prompt_32k", op="write", n=32768, Hq=32, Hkv=8, page=64, dtype="bf16", fused=True, pad=0,
             far=32768),
        # a small model's decode with few requests: latency
        dict(name="attn_decode_4", op="attn", B=4, Hq=16, Hkv=8, prefix=1024, page=16, cached_lo=0, cached_hi=100,
             new=1, long=0, long_new=0, pad=0),
        # decode of the repository's batch of 16, a prefix of 8192 and answers of up to 2000 tokens
        dict(name="attn_decode_16", op="attn", B=16, Hq=32, Hkv=8, prefix=8192, page=16, cached_lo=1, cached_hi=2000,
             new=1, long=0, long_new=0, pad=0),
        # 40/8 heads, a prefix that ends inside a page, padded batch
        dict(name="attn_decode_61", op="attn", B=61, Hq=40, Hkv=8, prefix=5003, page=32, cached_lo=1, cached_hi=700,
             new=1, long=0, long_new=0, pad=3),
        # a full serving batch over a 32K prefix
        dict(name="attn_decode_128", op="attn", B=128, Hq=32, Hkv=8, prefix=32768, page=64, cached_lo=1,
             cached_hi=2047, new=1, long=0, long_new=0, pad=0),
        # three proposed tokens for each request, checked in one pass
        dict(name="attn_verify_32", op="attn", B=32, Hq=32, Hkv=8, prefix=4096, page=16, cached_lo=10,
             cached_hi=1500, new=3, long=0, long_new=0, pad=0),
        # decodes with one request's prompt chunk among them
        dict(name="attn_mixed_8", op="attn", B=8, Hq=32, Hkv=8, prefix=4096, page=16, cached_lo=0, cached_hi=900,
             new=1, long=1, long_new=1000, pad=0),
        # four requests' own prompts behind the shared prefix
        dict(name="attn_prompt_4x1k", op="attn", B=4, Hq=32, Hkv=8, prefix=8192, page=64, cached_lo=0, cached_hi=0,
             new=1024, long=0, long_new=0, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        at = most.setdefault(c["op"], {"bytes": 0, "flops": 0})
        for k in at:
            at[k] = max(at[k], w[k])
    while True:
        op = rng.choice(["tables", "write", "attn", "attn"])
        page = rng.choice([16, 32, 64, 128])
        pad = rng.choice([0, 0, rng.randint(1, 40)])
        if op == "tables":
            B = _log(rng, 1, 256)
            long = rng.choice([0, rng.randint(0, B)])
            c = dict(op=op, B=B, page=page, cached_lo=rng.choice([0, 1, 17]), cached_hi=_log(rng, 20, 8192),
                     new=rng.choice([1, 1, 2, 5]), long=long, long_new=_log(rng, 2, 4000) if long else 0, pad=pad,
                     base=rng.choice([0, 1024, 8192]))
        elif op == "write":
            Hq, Hkv = rng.choice([(4, 2), (16, 8), (32, 8), (40, 8), (8, 8), (64, 8)])
            c = dict(op=op, n=_log(rng, 1, 32768), Hq=Hq, Hkv=Hkv, page=page, dtype=rng.choice(["bf16", "f32"]),
                     fused=rng.random() < 0.5, pad=pad, far=rng.choice([40000, 300000, 1 << 20]))
        else:
            Hq, Hkv = rng.choice([(4, 2), (16, 8), (32, 8), (40, 8), (8, 8), (64, 8)])
            B = _log(rng, 1, 128)
            kind = rng.choice(["decode", "decode", "verify", "mixed", "prompt"])
            long, long_new, new = 0, 0, 1
            if kind == "verify":
                new = rng.randint(2, 8)
            elif kind == "mixed":
                B = min(B, 16)
                long, long_new = rng.randint(1, max(1, B // 4)), _log(rng, 20, 1000)
            elif kind == "prompt":
                B = min(B, 8)
                new = _log(rng, 10, 1024)
            c = dict(op=op, B=B, Hq=Hq, Hkv=Hkv, prefix=rng.choice([0] + [_log(rng, 100, 32768)] * 7), page=page,
                     cached_lo=rng.choice([0, 1, 5]), cached_hi=_log(rng, 5, 2047), new=new, long=long,
                     long_new=long_new, pad=pad)
            mx = max(new, long_new)
            scores = 4 * Hq * (_total(c) * c["prefix"] + B * mx * (c["cached_hi"] + mx))
            if scores > 6 << 30:  # the plain form keeps its scores
                continue
        w = work(c)
        if all(w[k] <= most[op][k] for k in w):
            return c


def _lengths(case):
    """(tokens cached, tokens new) of each request, in the case's own order."""
    B, lo, hi = case["B"], case["cached_lo"], case["cached_hi"]
    at = np.arange(B) / max(1, B - 1)
    cached = np.rint(lo + (hi - lo) * at ** 2).astype(np.int64)
    new = np.full(B, case["new"], np.int64)
    if case["long"]:
        new[np.linspace(0, B - 1, case["long"]).astype(int)] = case["long_new"]
    return cached, new


def _total(case):
    return int(_lengths(case)[1].sum())


def work(case):
    if case["op"] == "tables":
        cached, new = _lengths(case)
        P, n = case["page"], int(new.sum())
        added = int((-(-(cached + new) // P) + -cached // P).sum())
        # lengths in; page ids taken and stored; slot and position of every row; offsets and lengths out
        return {"bytes": 16 * case["B"] + 8 * added + 12 * (n + case["pad"]), "flops": 0}
    if case["op"] == "write":
        e = 2 if case["dtype"] == "bf16" else 4
        rows = case["n"] * D
        heads, kv = case["Hq"] + 2 * case["Hkv"], 2 * case["Hkv"]
        return {"bytes": rows * (heads * e + case["Hq"] * 2 + kv * 2) + 12 * (case["n"] + case["pad"]),
                "flops": 6 * rows * (case["Hq"] + case["Hkv"])}
    cached, new = _lengths(case)
    n, S = int(new.sum()), cached + new
    keys = case["prefix"] + int(S.sum())
    pairs = n * case["prefix"] + int((new * cached + new * (new + 1) // 2).sum())
    return {"bytes": keys * case["Hkv"] * D * 2 * 2 + n * case["Hq"] * (2 * D * 2 + 4),
            "flops": 4 * D * case["Hq"] * pairs}


# -- inputs ----------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _dealt(case, seed):
    cached, new = _lengths(case)
    order = np.random.RandomState(seed & 0x7FFFFFFF).permutation(case["B"])
    return cached[order], new[order]


def _offsets(new):
    return np.concatenate([[0], np.cumsum(new)])


def _inputs_tables(case, seed):
    cached, new = _dealt(case, seed)
    P, B = case["page"], case["B"]
    have, need = -(-cached // P), -(-(cached + new) // P)
    rs = np.random.RandomState((seed * 7 + 1) & 0x7FFFFFFF)
    n_pages = int(need.sum()) + 50
    ids = rs.permutation(n_pages).astype(np.int32)
    table = np.full((B, int(need.max()) + 3), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, : have[b]] = ids[at: at + have[b]]
        at += have[b]
    return dict(case=case, P=P, n_pages=n_pages, cached=_i32(cached), new=_i32(new), rows=int(new.sum()) + case["pad"],
                free=_i32(ids), used=_i32([at]), table=_i32(table), base=case["base"])


def _inputs_write(case, seed):
    g, n = _gen(seed), case["n"]
    Hq, Hkv, P = case["Hq"], case["Hkv"], case["page"]
    rows = n + case["pad"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    x = torch.randn((rows, Hq + 2 * Hkv, D), generator=g, device="cuda").to(dt)
    q, k, v = x[:, :Hq], x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:]
    if not case["fused"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    n_pages = -(-n // P) + 4
    perm = torch.randperm(n_pages, generator=g, device="cuda")
    first = int(seed) % P  # the chunk begins inside a page
    at = torch.arange(first, first + n, device="cuda")
    slots = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
    slots[:n] = perm[at // P] * P + at % P
    pos = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    begin = max(0, case["far"] - n - int(seed) % 1000)
    pos[:n] = torch.arange(begin, begin + n, device="cuda", dtype=torch.int32)
    pool = [torch.randn((n_pages, Hkv, P, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    return dict(case=case, P=P, n=n, q=q, k=k, v=v, slots=slots, pos=pos, pages_k=pool[0], pages_v=pool[1],
                q_out=torch.zeros((rows, Hq, D), dtype=torch.bfloat16, device="cuda"))


def _inputs_attn(case, seed):
    g = _gen(seed)
    cached, new = _dealt(case, seed)
    Hq, Hkv, P, B = case["Hq"], case["Hkv"], case["page"], case["B"]
    lens, n = cached + new, int(new.sum())
    own_pages, shared = -(-lens // P), -(-case["prefix"] // P)
    n_pages = shared + int(own_pages.sum()) + 2
    ids = np.random.RandomState((seed * 7 + 1) & 0x7FFFFFFF).permutation(n_pages).astype(np.int32)
    table = np.full((B, max(1, int(own_pages.max()))), -1, np.int32)
    at = shared
    for b in range(B):
        table[b, : own_pages[b]] = ids[at: at + own_pages[b]]
        at += own_pages[b]
    # keys with channels of unequal size, as rotary models have them, and queries that single some keys out
    size = torch.exp(0.4 * torch.randn((1, Hkv, 1, D), generator=g, device="cuda"))
    k = torch.randn((n_pages, Hkv, P, D), generator=g, device="cuda", dtype=torch.bfloat16).mul_(size.bfloat16())
    v = torch.randn((n_pages, Hkv, P, D), generator=g, device="cuda", dtype=torch.bfloat16)
    rows = n + case["pad"]
    q = (1.5 * torch.randn((rows, Hq, D), generator=g, device="cuda")).to(torch.bfloat16)
    return dict(case=case, P=P, n=n, mx=int(new.max()), q=q, pages_k=k, pages_v=v, table=_i32(table),
                q_start=_i32(_offsets(new)), lens=_i32(lens), prefix=_i32(ids[:shared]), prefix_len=case["prefix"],
                out=torch.zeros((rows, Hq, D), dtype=torch.bfloat16, device="cuda"),
                lse=torch.zeros((rows, Hq), dtype=torch.float32, device="cuda"))


def _inputs(case, seed):
    return {"tables": _inputs_tables, "write": _inputs_write, "attn": _inputs_attn}[case["op"]](case, seed)


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "tables":
        B, rows = case["B"], s["rows"]
        s["slots"] = torch.zeros(rows, dtype=torch.int64, device="cuda")
        s["pos"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
        s["q_start"] = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        s["lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        s["used_out"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        import hierarchical_kv_cache_hsq_gb300 as H
        Hq, Hkv, B = case.get("Hq", 1), case.get("Hkv", 1), case.get("B", 1)
        s["ctx"] = ctx = H.Context(H.make_config(Hq, Hkv, 16, 1, B, 16, 0, case.get("far", 16), theta=THETA))
        if case["op"] == "tables":
            s["pool"] = H.allocate_pages(ctx, s["n_pages"], s["P"])
        else:
            s["pool"] = H.PagePool(s["pages_k"], s["pages_v"])
        if case["op"] == "attn":
            need = H.hsq_shared_attn_workspace_size(ctx, s["q"].shape[0], B, s["prefix_len"], s["mx"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# -- one pass -----------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        import hierarchical_kv_cache_hsq_gb300 as H
        if op == "tables":
            H.hsq_page_tables(s["ctx"], s["pool"], s["cached"], s["new"], s["free"], s["used"], s["table"], s["slots"],
                              s["pos"], s["q_start"], s["lens"], s["used_out"], base=s["base"])
        elif op == "write":
            H.hsq_page_write(s["ctx"], s["pool"], s["q"], s["k"], s["v"], s["pos"], s["slots"], s["q_out"])
        else:
            H.hsq_shared_attn(s["ctx"], s["pool"], s["q"], s["q_start"], s["lens"], s["table"], s["out"],
                              s["workspace"], prefix=s["prefix"], prefix_len=s["prefix_len"], max_new=s["mx"],
                              lse=s["lse"])
    else:
        {"tables": _plain_tables, "write": _plain_write, "attn": _plain_attn}[op](s)
    if op == "tables":
        return {k: s[k] for k in ("table", "slots", "pos", "q_start", "lens", "used_out")}
    if op == "write":
        return {k: s[k] for k in ("q_out", "pages_k", "pages_v")}
    return {"out": s["out"], "lse": s["lse"]}


def _plain_tables(s):
    P, table, free = s["P"], s["table"], s["free"]
    cached, new = s["cached"].long(), s["new"].long()
    lens = cached + new
    have, need = (cached + P - 1) // P, (lens + P - 1) // P
    added = need - have
    end = torch.cumsum(added, 0)
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    at = s["used"].long() + (end - added)[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    ids = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], -1)
    table.copy_(torch.where(fresh, ids, table))
    stop = torch.cumsum(new, 0)
    s["q_start"][1:] = stop
    s["lens"].copy_(lens)
    s["used_out"].copy_(torch.clamp(s["used"].long() + end[-1:], max=free.numel()))
    row = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(stop, row, right=True).clamp(max=new.numel() - 1)
    p = cached[b] + row - (stop - new)[b]
    live = row < stop[-1]
    page = table[b, (p // P).clamp(0, table.shape[1] - 1)].long()
    s["slots"].copy_(torch.where(live & (page >= 0), page * P + p % P, -1))
    s["pos"].copy_(torch.where(live, s["base"] + p, -1))


def _rotated(x, pos):
    """Rotate-half of x [n, heads, 128] at pos: the angles in 64 bits, the products in 32."""
    w = THETA ** (-2.0 * torch.arange(D // 2, device="cuda", dtype=torch.float64) / D)
    a = pos.double()[:, None] * w[None, :]
    c, s = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    lo, hi = x[..., : D // 2].float(), x[..., D // 2:].float()
    return torch.cat([lo * c - hi * s, hi * c + lo * s], dim=-1)


def _plain_write(s):
    n, P = s["n"], s["P"]
    pos, slots = s["pos"][:n], s["slots"][:n]
    s["q_out"][:n] = _rotated(s["q"][:n], pos).bfloat16()
    s["pages_k"][slots // P, :, slots % P] = _rotated(s["k"][:n], pos).bfloat16()
    s["pages_v"][slots // P, :, slots % P] = s["v"][:n].bfloat16()


def _part(q, k, v, seen):
    """Softmax parts of q [..., rows, 128] over k, v [..., keys, 128]: maxima, sums, weighted values."""
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(D ** -0.5)
    if seen is not None:
        x.masked_fill_(~seen, -float("inf"))
    m = x.amax(-1)
    x.sub_(m.clamp(min=-1e30)[..., None]).exp_()
    return m, x.sum(-1), torch.matmul(x, v)


def _plain_attn(s):
    n, P, mx = s["n"], s["P"], s["mx"]
    Hkv, Hq = s["pages_k"].shape[1], s["q"].shape[1]
    r, B, W = Hq // Hkv, s["lens"].numel(), s["table"].shape[1]
    q = s["q"][:n].float().view(n, Hkv, r, D)
    start, lens = s["q_start"][:-1].long(), s["lens"].long()
    new = s["q_start"][1:].long() - start
    # every request's own keys, its rows side by side
    j = torch.arange(mx, device="cuda")[None, :]
    rows = (start[:, None] + j).clamp(max=n - 1)
    at = torch.arange(W * P, device="cuda")
    ids = s["table"].long().clamp(min=0)
    have = (at[None, :] < lens[:, None])[:, None, :, None]
    ko = s["pages_k"][ids].transpose(1, 2).reshape(B, Hkv, W * P, D).float().masked_fill_(~have, 0)
    vo = s["pages_v"][ids].transpose(1, 2).reshape(B, Hkv, W * P, D).float().masked_fill_(~have, 0)
    last = (lens - new)[:, None] + j
    seen = (at[None, None, :] <= last[:, :, None]) & (at[None, None, :] < lens[:, None, None])
    seen = seen[:, None, :, None, :].expand(B, 1, mx, r, W * P).reshape(B, 1, mx * r, W * P)
    qo = q[rows].permute(0, 2, 1, 3, 4).reshape(B, Hkv, mx * r, D)
    mo, lo, ao = _part(qo, ko, vo, seen)
    of_row = torch.arange(n, device="cuda")
    b = torch.searchsorted(s["q_start"][1:].long(), of_row, right=True)
    jj = of_row - start[b]
    m = mo.view(B, Hkv, mx, r)[b, :, jj]
    l = lo.view(B, Hkv, mx, r)[b, :, jj]
    a = ao.view(B, Hkv, mx, r, D)[b, :, jj]
    if s["prefix_len"]:
        ids = s["prefix"].long()
        kp = s["pages_k"][ids].transpose(0, 1).reshape(Hkv, -1, D)[:, : s["prefix_len"]].float()
        vp = s["pages_v"][ids].transpose(0, 1).reshape(Hkv, -1, D)[:, : s["prefix_len"]].float()
        mp, lp, ap = _part(q.transpose(0, 1).reshape(Hkv, n * r, D), kp, vp, None)
        mp, lp = mp.view(Hkv, n, r).transpose(0, 1), lp.view(Hkv, n, r).transpose(0, 1)
        ap = ap.view(Hkv, n, r, D).transpose(0, 1)
        top = torch.maximum(m, mp)
        wo, wp = torch.exp(m - top), torch.exp(mp - top)
        m, l, a = top, l * wo + lp * wp, a * wo[..., None] + ap * wp[..., None]
    s["out"][:n] = (a / l[..., None]).view(n, Hq, D).bfloat16()
    s["lse"][:n] = (m + torch.log(l)).view(n, Hq)


# -- the operators' definition in 64 bits ------------------------------------------------------

def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = _inputs(case, seed)
    n, P = s["n"], s["P"]
    if case["op"] == "write":
        pos, slots = s["pos"][:n].cpu().numpy().astype(np.float64), s["slots"][:n].cpu().numpy()
        ang = pos[:, None] * np.power(THETA, -np.arange(0, D, 2) / D)[None, :]
        turn = torch.from_numpy(np.exp(1j * ang)).cuda()[:, None, :]

        def rot(x):
            z = torch.complex(x[..., : D // 2].double(), x[..., D // 2:].double()) * turn
            return torch.cat([z.real, z.imag], -1)

        q_out = torch.zeros(s["q_out"].shape, dtype=torch.float64, device="cuda")
        q_out[:n] = rot(s["q"][:n])
        pk, pv = s["pages_k"].double(), s["pages_v"].double()
        page, off = torch.from_numpy(slots // P).cuda(), torch.from_numpy(slots % P).cuda()
        pk[page, :, off] = rot(s["k"][:n])
        pv[page, :, off] = s["v"][:n].double()
        return {"q_out": q_out, "pages_k": pk, "pages_v": pv}
    Hq, Hkv = case["Hq"], case["Hkv"]
    r = Hq // Hkv
    rows = n + case["pad"]
    out = torch.zeros((rows, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((rows, Hq), dtype=torch.float64, device="cuda")
    start, lens = s["q_start"].tolist(), s["lens"].tolist()

    def tokens(pages, ids, count, h):
        return pages[ids[: -(-count // P)].long(), h].reshape(-1, D)[:count].double()

    for h in range(Hkv):  # one softmax over the prefix's keys and the request's own
        kp, vp = tokens(s["pages_k"], s["prefix"], s["prefix_len"], h), tokens(s["pages_v"], s["prefix"], s["prefix_len"], h)
        for b in range(case["B"]):
            a, e = start[b], start[b + 1]
            k = torch.cat([kp, tokens(s["pages_k"], s["table"][b], lens[b], h)])
            v = torch.cat([vp, tokens(s["pages_v"], s["table"][b], lens[b], h)])
            x = s["q"][a:e, h * r: (h + 1) * r].double().reshape(-1, D) @ k.T / D ** 0.5
            limit = s["prefix_len"] + lens[b] - (e - a) + torch.arange(e - a, device="cuda").repeat_interleave(r)
            x = x.masked_fill(torch.arange(k.shape[0], device="cuda")[None, :] > limit[:, None], -float("inf"))
            z = torch.logsumexp(x, -1)
            out[a:e, h * r: (h + 1) * r] = (torch.exp(x - z[:, None]) @ v).view(e - a, r, D)
            lse[a:e, h * r: (h + 1) * r] = z.view(e - a, r)
    return {"out": out, "lse": lse}
