"""What is measured of the long-context operators over the page pool: the paged
write with a model's own rotation (interleaved or half layout, part of the
head, scaled for long contexts), the pages' 8-bit summaries, the selection of
pages by a cheap score for every row and KV head, and the attention over the
selected pages alone.

A serving step over a long context calls them in that order.  Request b's
logical pages are those of the shared prefix, then its own; a selection names
logical pages.  As in earlier serving cases, a case's request lengths are one
fixed list, dealt to the requests in an order that the seed decides.
"""

import math

import numpy as np
import torch

own = False

D = 128
THETA = 1.0e6
FIRST, RECENT = 1, 2  # pages that every row takes: the context's first one, its last two


# -- cases ---------------------------------------------------------------------------

def listed():
    return [
        # the new tokens of a decode step, 32/8 heads, frequencies ramped for four times the original context
        dict(name="rotate_decode_16", op="rotate", n=16, Hq=32, Hkv=8, page=16, dtype="bf16", fused=True, pad=0,
             dims=128, pairs="half", scaling="yarn", factor=4.0, far=131072),
        # a float32 model's odd-sized chunk, 40/8 heads, half of the head rotated in neighbouring pairs
        dict(name="rotate_chunk_f32", op="rotate", n=2531, Hq=40, Hkv=8, page=128, dtype="f32", fused=False, pad=29,
             dims=64, pairs="neighbours", scaling="linear", factor=8.0, far=1 << 20),
        # a whole prompt, views of one fused projection, neighbouring pairs over the whole head
        dict(name="rotate_prompt_32k", op="rotate", n=32768, Hq=32, Hkv=8, page=64, dtype="bf16", fused=True, pad=0,
             dims=128, pairs="neighbours", scaling="base", factor=2.0, far=65536),
        # the pages that a decode step of 16 requests touches
        dict(name="sums_decode_16", op="sums", B=16, Hkv=8, page=16, new=1, pad=0),
        # the pages of a whole prompt
        dict(name="sums_prompt_32k", op="sums", B=1, Hkv=8, page=64, new=32768, pad=100),
        # decode of 16 requests behind a prefix of 8192, up to 2048 small pages each
        dict(name="select_decode_16", op="select", B=16, Hq=32, Hkv=8, prefix=8192, page=16, cached_lo=100,
             cached_hi=24575, new=1, long=0, long_new=0, pad=0, top=64),
        # four requests at 128K tokens each
        dict(name="select_decode_128k", op="select", B=4, Hq=32, Hkv=8, prefix=0, page=32, cached_lo=100000,
             cached_hi=131071, new=1, long=0, long_new=0, pad=3, top=128),
        # a prompt's chunk of 2048 tokens at the end of 32K
        dict(name="select_prompt_2k", op="select", B=1, Hq=32, Hkv=8, prefix=0, page=32, cached_lo=30720,
             cached_hi=30720, new=2048, long=0, long_new=0, pad=0, top=64),
        # a small model's decode with few requests: latency
        dict(name="attn_decode_4", op="attn", B=4, Hq=16, Hkv=8, prefix=1000, page=16, cached_lo=10, cached_hi=7000,
             new=1, long=0, long_new=0, pad=0, top=16),
        # decode of a full batch, 2048 of up to 20K tokens for each row and head
        dict(name="attn_decode_64", op="attn", B=64, Hq=32, Hkv=8, prefix=4096, page=64, cached_lo=2000,
             cached_hi=16384, new=1, long=0, long_new=0, pad=5, top=32),
        # five proposed tokens of each request, 40/8 heads, checked in one pass
        dict(name="attn_verify_24", op="attn", B=24, Hq=40, Hkv=8, prefix=0, page=16, cached_lo=500, cached_hi=9001,
             new=5, long=0, long_new=0, pad=0, top=64),
        # a prompt's chunk of 2048 tokens at the end of 32K
        dict(name="attn_prompt_2k", op="attn", B=1, Hq=32, Hkv=8, prefix=0, page=32, cached_lo=30720,
             cached_hi=30720, new=2048, long=0, long_new=0, pad=0, top=64),
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
        op = rng.choice(["rotate", "sums", "select", "select", "attn", "attn", "attn"])
        page = rng.choice([16, 32, 64, 128])
        pad = rng.choice([0, 0, rng.randint(1, 40)])
        Hq, Hkv = rng.choice([(4, 2), (16, 8), (32, 8), (40, 8), (8, 8), (64, 8)])
        if op == "rotate":
            far = rng.choice([40000, 300000, 1 << 20])
            c = dict(op=op, n=_log(rng, 1, 32768), Hq=Hq, Hkv=Hkv, page=page, dtype=rng.choice(["bf16", "f32"]),
                     fused=rng.random() < 0.5, pad=pad, dims=rng.choice([32, 64, 96, 128]),
                     pairs=rng.choice(["half", "neighbours"]), scaling=rng.choice(["none", "linear", "base", "yarn"]),
                     factor=rng.choice([2.0, 4.0, 32.0]), far=far)
        elif op == "sums":
            B = _log(rng, 1, 64)
            c = dict(op=op, B=B, Hkv=Hkv, page=page, new=rng.choice([1, rng.randint(2, 8), _log(rng, 1, 32768 // B)]),
                     pad=pad)
        else:
            B = _log(rng, 1, 64)
            kind = rng.choice(["decode", "decode", "verify", "mixed", "prompt"])
            long, long_new, new = 0, 0, 1
            if kind == "verify":
                new = rng.randint(2, 8)
            elif kind == "mixed":
                B = min(B, 8)
                long, long_new = rng.randint(1, max(1, B // 4)), _log(rng, 20, 1000)
            elif kind == "prompt":
                B = min(B, 3)
                new = _log(rng, 10, 2048)
            c = dict(op=op, B=B, Hq=Hq, Hkv=Hkv, prefix=rng.choice([0, 0, _log(rng, 100, 8192)]), page=page,
                     cached_lo=rng.choice([0, 1, 900]), cached_hi=_log(rng, 1000, 32768 if B > 4 else 131072),
                     new=new, long=long, long_new=long_new, pad=pad, top=rng.choice([4, 16, 37, 64, 128]))
            mx = max(new, long_new)
            pages = (c["prefix"] + c["cached_hi"] + mx) / page
            if B * mx * Hkv * pages > 1 << 28 or B * (c["cached_hi"] + mx) > 1 << 20:
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


def work(case):
    if case["op"] == "rotate":
        e = 2 if case["dtype"] == "bf16" else 4
        rows = case["n"] * D
        heads, kv = case["Hq"] + 2 * case["Hkv"], 2 * case["Hkv"]
        return {"bytes": rows * (heads * e + case["Hq"] * 2 + kv * 2) + 12 * (case["n"] + case["pad"]),
                "flops": 6 * case["n"] * case["dims"] * (case["Hq"] + case["Hkv"])}
    if case["op"] == "sums":
        n = case["B"] * case["new"]
        pages = case["B"] * -(-case["new"] // case["page"])
        keys = max(n, pages)  # a page is read as far as it is filled
        return {"bytes": case["Hkv"] * (keys * D * 2 + pages * (D + 4)) + 8 * (n + case["pad"]),
                "flops": case["Hkv"] * keys * D}
    cached, new = _lengths(case)
    n, P, pre = int(new.sum()), case["page"], case["prefix"]
    shared = -(-pre // P)
    mean_own = cached + (new + 1) / 2  # own tokens that a row sees, on average
    if case["op"] == "select":
        pages = shared + int((-(-(cached + new) // P)).sum())
        pairs = case["Hkv"] * int((new * (shared + mean_own / P)).sum())
        return {"bytes": pages * case["Hkv"] * (D + 4) + n * (case["Hq"] * D * 2 + case["Hkv"] * case["top"] * 4),
                "flops": 2 * D * pairs}
    keys = np.minimum(case["top"] * P, pre + cached + new)  # at least what its last row attends to
    seen = np.minimum(case["top"] * P, pre + mean_own)
    return {"bytes": int(keys.sum()) * case["Hkv"] * D * 2 * 2 +
            n * (case["Hq"] * (2 * D * 2 + 4) + case["Hkv"] * case["top"] * 4),
            "flops": int(4 * D * case["Hq"] * float((new * seen).sum()))}


# -- inputs ----------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _freqs(case):
    """The pairs' frequencies (float64) and the amplitude of the rotated parts."""
    R, kind, f = case["dims"], case["scaling"], case["factor"]
    i = np.arange(R // 2)
    theta = THETA * f ** (R / (R - 2)) if kind == "base" else THETA
    w, amp = theta ** (-2.0 * i / R), 1.0
    if kind == "linear":
        w = w / f
    elif kind == "yarn":
        turns = (case["far"] / f) * w / (2 * math.pi)  # over the original context
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        w, amp = w * (keep + (1 - keep) / f), 0.1 * math.log(f) + 1.0
    return w, amp


def _inputs_rotate(case, seed):
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


def _inputs_sums(case, seed):
    """The slots of a step's rows: each request's tokens go on inside a page and fill the pages after it."""
    g, B, new, P, Hkv = _gen(seed), case["B"], case["new"], case["page"], case["Hkv"]
    rs = np.random.RandomState((seed * 7 + 1) & 0x7FFFFFFF)
    first = rs.randint(0, P, B)
    used = -(-(first + new) // P)
    n_pages = B * -(-(P - 1 + new) // P) + 3
    ids = rs.permutation(n_pages)
    slots, at = np.full(B * new + case["pad"], -1, np.int64), 0
    for b in range(B):
        t = first[b] + np.arange(new)
        slots[b * new: (b + 1) * new] = ids[at + t // P] * P + t % P
        at += used[b]
    size = torch.exp(0.4 * torch.randn((1, Hkv, 1, D), generator=g, device="cuda"))
    k = torch.randn((n_pages, Hkv, P, D), generator=g, device="cuda")
    k = ((k + torch.randn((n_pages, Hkv, 1, D), generator=g, device="cuda")) * size).to(torch.bfloat16)
    codes = torch.randint(-127, 128, (n_pages, Hkv, D), generator=g, device="cuda", dtype=torch.int8)
    scale = torch.rand((n_pages, Hkv), generator=g, device="cuda")
    return dict(case=case, P=P, slots=torch.from_numpy(slots).cuda(), pages_k=k, codes=codes, scale=scale)


def _inputs_context(case, seed, values):
    """A pool whose tokens go from topic to topic, and queries that look for some of the topics: what
    makes a few pages matter, and neighbouring rows mostly the same ones."""
    g = _gen(seed)
    rs = np.random.RandomState((seed * 7 + 1) & 0x7FFFFFFF)
    cached, new = _lengths(case)
    order = np.random.RandomState(seed & 0x7FFFFFFF).permutation(case["B"])
    cached, new = cached[order], new[order]
    Hq, Hkv, P, B, pre = case["Hq"], case["Hkv"], case["page"], case["B"], case["prefix"]
    lens, n = cached + new, int(new.sum())
    own_pages, shared = -(-lens // P), -(-pre // P)
    n_pages = shared + int(own_pages.sum()) + 2
    ids = rs.permutation(n_pages).astype(np.int32)
    table = np.full((B, max(1, int(own_pages.max()))), -1, np.int32)
    topic = np.zeros((n_pages, P), np.int64)  # of the pool's tokens
    span = 96
    topic[ids[:shared]] = (np.arange(shared * P) // span).reshape(shared, P)
    ends, at, topics = [], shared, -(-shared * P // span)
    for b in range(B):
        table[b, : own_pages[b]] = ids[at: at + own_pages[b]]
        topic[table[b, : own_pages[b]]] = topics + (np.arange(own_pages[b] * P) // span).reshape(-1, P)
        ends.append((topics, topics + -(-int(lens[b]) // span)))
        topics += -(-int(own_pages[b]) * P // span) + 1
        at += own_pages[b]
    size = torch.exp(0.4 * torch.randn((1, Hkv, 1, D), generator=g, device="cuda"))
    themes = torch.randn((topics + 1, Hkv, D), generator=g, device="cuda")
    topic = torch.from_numpy(topic).cuda()
    k = torch.empty((n_pages, Hkv, P, D), dtype=torch.bfloat16, device="cuda")
    for a in range(0, n_pages, 4096):
        part = themes[topic[a: a + 4096]].transpose(1, 2)
        k[a: a + 4096] = (size * (part + torch.randn(part.shape, generator=g, device="cuda"))).to(torch.bfloat16)
    v = torch.randn(k.shape, generator=g, device="cuda", dtype=torch.bfloat16) if values else k
    # rows: every 48 tokens of a request look for six topics that lie behind them
    rows = n + case["pad"]
    look = np.zeros((n, 6), np.int64)
    i = 0
    in_prefix = -(-pre // span)
    for b in range(B):
        for j0 in range(0, int(new[b]), 48):
            j1 = min(j0 + 48, int(new[b]))
            behind = in_prefix + max(1, int(cached[b] + j0) // span)
            pick = rs.randint(0, behind, 6)
            look[i: i + j1 - j0] = np.where(pick < in_prefix, pick, ends[b][0] + pick - in_prefix)
            i += j1 - j0
    want = themes[torch.from_numpy(look).cuda()].mean(1) * 0.7
    q = torch.zeros((rows, Hq, D), dtype=torch.bfloat16, device="cuda")
    noise = 0.6 * torch.randn((n, Hkv, Hq // Hkv, D), generator=g, device="cuda")
    q[:n] = (want[:, :, None] + noise).view(n, Hq, D).to(torch.bfloat16)
    start = np.concatenate([[0], np.cumsum(new)])
    return dict(case=case, P=P, n=n, mx=int(new.max()), q=q, pages_k=k, pages_v=v, table=_i32(table),
                q_start=_i32(start), lens=_i32(lens), prefix=_i32(ids[:shared]), prefix_len=pre,
                sel=torch.full((rows, Hkv, case["top"]), -1, dtype=torch.int32, device="cuda"))


def _inputs_select(case, seed):
    s = _inputs_context(case, seed, False)
    s["codes"], s["scale"] = _summed(s["pages_k"], torch.full((s["pages_k"].shape[0],), s["P"], device="cuda"))
    return s


def _inputs_attn(case, seed):
    s = _inputs_context(case, seed, True)
    s["codes"], s["scale"] = _summed(s["pages_k"], torch.full((s["pages_k"].shape[0],), s["P"], device="cuda"))
    _plain_select(s)
    del s["codes"], s["scale"]
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    return s


def _inputs(case, seed):
    return {"rotate": _inputs_rotate, "sums": _inputs_sums, "select": _inputs_select, "attn": _inputs_attn}[
        case["op"]](case, seed)


def prepare(case, seed):
    s, op = _inputs(case, seed), case["op"]
    if own:
        import hierarchical_kv_cache_hsq_gb300 as H
        Hkv = case["Hkv"]
        far = case.get("far", 16)
        s["ctx"] = ctx = H.Context(H.make_config(case.get("Hq", Hkv), Hkv, 16, 1, case.get("B", 1), 16, 0, far,
                                                 theta=THETA))
        s["pool"] = pool = H.PagePool(s["pages_k"], s.get("pages_v", s["pages_k"]))
        if op == "rotate":
            s["rope"] = H.make_rope(ctx, dims=case["dims"], interleaved=case["pairs"] == "neighbours",
                                    scaling=case["scaling"], factor=case["factor"],
                                    original=case["far"] / case["factor"])
        else:
            if op != "attn":
                s["sums"] = H.PageSummaries(s["codes"], s["scale"])
            if op != "sums":
                size = H.hsq_page_select_workspace_size if op == "select" else H.hsq_page_attn_workspace_size
                need = size(ctx, pool, s["q"].shape[0], case["B"], s["table"].shape[1], s["prefix_len"], case["top"],
                            s["mx"])
                s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# -- one pass -----------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        import hierarchical_kv_cache_hsq_gb300 as H
        if op == "rotate":
            H.hsq_page_write(s["ctx"], s["pool"], s["q"], s["k"], s["v"], s["pos"], s["slots"], s["q_out"],
                             rope=s["rope"])
        elif op == "sums":
            H.hsq_page_summaries(s["ctx"], s["pool"], s["sums"], s["slots"])
        elif op == "select":
            H.hsq_page_select(s["ctx"], s["pool"], s["sums"], s["q"], s["q_start"], s["lens"], s["table"], s["sel"],
                              s["workspace"], prefix=s["prefix"], prefix_len=s["prefix_len"], first=FIRST,
                              recent=RECENT, max_new=s["mx"])
        else:
            H.hsq_page_attn(s["ctx"], s["pool"], s["q"], s["q_start"], s["lens"], s["table"], s["sel"], s["out"],
                            s["workspace"], prefix=s["prefix"], prefix_len=s["prefix_len"], max_new=s["mx"],
                            lse=s["lse"])
    else:
        {"rotate": _plain_rotate, "sums": _plain_sums, "select": _plain_select, "attn": _plain_attn}[op](s)
    if op == "rotate":
        return {k: s[k] for k in ("q_out", "pages_k", "pages_v")}
    if op == "sums":  # the values that the codes stand for
        return s["codes"] * s["scale"][..., None]
    if op == "select":
        return s["sel"]
    return {"out": s["out"], "lse": s["lse"]}


def _rotated(x, pos, case):
    """x [n, heads, 128] rotated at pos: the angles in 64 bits, the products in 32."""
    R = case["dims"]
    w, amp = _freqs(case)
    a = pos.double()[:, None] * torch.from_numpy(w).cuda()[None, :]
    c, s = (amp * torch.cos(a)).float()[:, None], (amp * torch.sin(a)).float()[:, None]
    out = x.float().clone()
    if case["pairs"] == "half":
        lo, hi = x[..., : R // 2].float(), x[..., R // 2: R].float()
        out[..., : R // 2], out[..., R // 2: R] = lo * c - hi * s, hi * c + lo * s
    else:
        lo, hi = x[..., 0: R: 2].float(), x[..., 1: R: 2].float()
        out[..., 0: R: 2], out[..., 1: R: 2] = lo * c - hi * s, hi * c + lo * s
    return out


def _plain_rotate(s):
    n, P, case = s["n"], s["P"], s["case"]
    pos, slots = s["pos"][:n], s["slots"][:n]
    s["q_out"][:n] = _rotated(s["q"][:n], pos, case).bfloat16()
    s["pages_k"][slots // P, :, slots % P] = _rotated(s["k"][:n], pos, case).bfloat16()
    s["pages_v"][slots // P, :, slots % P] = s["v"][:n].bfloat16()


def _codes(x):
    """8-bit codes of x [..., 128] (float32), 0 where it has no direction."""
    top = x.abs().amax(-1)
    live = torch.isfinite(top) & (top >= 2.0 ** -64)
    by = torch.full_like(top, 127.0) / torch.where(live, top, 1.0)
    return torch.where(live[..., None], torch.round(x * by[..., None]), 0.0)


def _summed(k, count):
    """Codes and scales of pages k [n, Hkv, P, 128] holding count [n] tokens: the sums in 64 bits, since a code
    changes by one at a border."""
    total = torch.zeros(k.shape[:2] + (D,), dtype=torch.float64, device="cuda")
    for t in range(k.shape[2]):
        total += torch.where((t < count)[:, None, None], k[:, :, t].double(), 0.0)
    top = total.abs().amax(-1)
    live = (top >= 2.0 ** -64) & (top <= 2.0 ** 126)
    codes = torch.where(live[..., None], torch.round(127.0 * total / torch.where(live, top, 1.0)[..., None]), 0.0)
    scale = top / (127.0 * count.double()[:, None])
    scale = torch.where(live, scale, torch.where(top < 2.0 ** -64, 0.0, float("inf")))
    return codes.to(torch.int8), scale.float()


def _plain_sums(s):
    P, slots = s["P"], s["slots"]
    after = torch.cat([slots[1:], torch.full((1,), -1, dtype=torch.int64, device="cuda")])
    last = (slots >= 0) & ((after < 0) | (after // P != slots // P))  # a page's last row of the step
    page, count = (slots // P)[last], (slots % P)[last] + 1
    s["codes"][page], s["scale"][page] = _summed(s["pages_k"][page], count)


def _logical(s):
    """Page ids [B, L] of the requests' logical pages, and each row's (request, own tokens seen)."""
    B = s["lens"].numel()
    ids = torch.cat([s["prefix"].long()[None, :].expand(B, -1), s["table"].long()], 1)
    row = torch.arange(s["n"], device="cuda")
    b = torch.searchsorted(s["q_start"][1:].long(), row, right=True)
    seen = s["lens"].long()[b] - s["q_start"].long()[b + 1] + row + 1
    return ids, b, seen


def _plain_select(s):
    case, n, P = s["case"], s["n"], s["P"]
    Hq, Hkv, top = case["Hq"], case["Hkv"], case["top"]
    ids, b, seen = _logical(s)
    shared, L = s["prefix"].numel(), ids.shape[1]
    x = s["q"][:n].view(n, Hkv, Hq // Hkv, D).float()
    total = x[:, :, 0]
    for j in range(1, Hq // Hkv):
        total = total + x[:, :, j]
    cq = _codes(total)
    col = torch.arange(L, device="cuda")
    starts = s["q_start"].tolist()
    for r in range(case["B"]):
        have = ids[r].clamp(min=0)
        cm, scale = s["codes"][have].float().permute(1, 2, 0), s["scale"][have].t()
        for a in range(starts[r], starts[r + 1], 512):
            e = min(a + 512, starts[r + 1])
            score = torch.matmul(cq[a:e].transpose(0, 1), cm) * scale[:, None, :]  # whole numbers below 2^24, one rounding
            pages = (shared + (seen[a:e] + P - 1) // P)[None, :, None]
            score = score.masked_fill((col < FIRST) | (col >= pages - RECENT), float("inf"))
            score = score.masked_fill(col >= pages, -float("inf"))
            at = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :top]
            at = torch.where(at < pages, at, L)
            at = torch.sort(at, dim=-1)[0]
            at = torch.where(at < L, at, -1).transpose(0, 1)
            s["sel"][a:e] = -1
            s["sel"][a:e, :, : at.shape[2]] = at.int()


def _plain_attn(s):
    case, n, P = s["case"], s["n"], s["P"]
    Hq, Hkv, top = case["Hq"], case["Hkv"], case["top"]
    ids, b, seen = _logical(s)
    shared = s["prefix"].numel()
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    step = max(1, (1 << 27) // (Hkv * top * P * D))
    for a in range(0, n, step):
        e = min(a + step, n)
        sel = s["sel"][a:e].long()
        page = ids[b[a:e, None, None], sel.clamp(min=0)]
        k = s["pages_k"][page, head].float().flatten(2, 3)
        v = s["pages_v"][page, head].float().flatten(2, 3)
        own = sel >= shared
        held = torch.where(own, seen[a:e, None, None] - (sel - shared) * P, s["prefix_len"] - sel * P)
        held = torch.where(sel >= 0, held, 0)
        ok = (torch.arange(P, device="cuda") < held[..., None]).flatten(2, 3)
        q = s["q"][a:e].float().view(e - a, Hkv, Hq // Hkv, D)
        x = torch.matmul(q, k.transpose(-1, -2)) * D ** -0.5
        x = x.masked_fill(~ok[:, :, None], -float("inf"))
        m = x.amax(-1, keepdim=True)
        w = torch.exp(x - m)
        l = w.sum(-1, keepdim=True)
        s["out"][a:e] = (torch.matmul(w, v) / l).view(e - a, Hq, D).bfloat16()
        s["lse"][a:e] = (m + torch.log(l)).view(e - a, Hq)


# -- the operators' definition in 64 bits ------------------------------------------------------

def exact(case, seed):
    if case["op"] == "select":
        return None  # whole numbers
    s = _inputs(case, seed)
    P = s["P"]
    if case["op"] == "rotate":
        n, R = s["n"], case["dims"]
        w, amp = _freqs(case)
        pos, slots = s["pos"][:n].cpu().numpy().astype(np.float64), s["slots"][:n].cpu().numpy()
        turn = torch.from_numpy(amp * np.exp(1j * pos[:, None] * w[None, :])).cuda()[:, None, :]
        even = slice(0, R, 2) if case["pairs"] == "neighbours" else slice(0, R // 2)
        odd = slice(1, R, 2) if case["pairs"] == "neighbours" else slice(R // 2, R)

        def rot(x):
            x = x.double()
            z = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * turn
            x = x.clone()
            x[..., even], x[..., odd] = z.real, z.imag
            return x

        q_out = torch.zeros(s["q_out"].shape, dtype=torch.float64, device="cuda")
        q_out[:n] = rot(s["q"][:n])
        pk, pv = s["pages_k"].double(), s["pages_v"].double()
        page, off = torch.from_numpy(slots // P).cuda(), torch.from_numpy(slots % P).cuda()
        pk[page, :, off] = rot(s["k"][:n])
        pv[page, :, off] = s["v"][:n].double()
        return {"q_out": q_out, "pages_k": pk, "pages_v": pv}
    if case["op"] == "sums":
        values = s["codes"].double() * s["scale"].double()[..., None]
        filled = {}
        for t in s["slots"].tolist():
            if t >= 0:
                filled.setdefault(t % P + 1, {})
                filled[t % P + 1][t // P] = True
        seen = {}
        for count in sorted(filled):
            for page in filled[count]:
                seen[page] = count  # the largest offset of the step
        for count in sorted(set(seen.values())):
            page = torch.tensor([p for p in seen if seen[p] == count], device="cuda")
            total = s["pages_k"][page, :, :count].double().sum(2)
            top = total.abs().amax(-1, keepdim=True)
            values[page] = torch.round(127 * total / top) * (top / (127 * count))
        return values
    Hq, Hkv = case["Hq"], case["Hkv"]
    r = Hq // Hkv
    rows = s["q"].shape[0]
    out = torch.zeros((rows, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((rows, Hq), dtype=torch.float64, device="cuda")
    start, lens, pre = s["q_start"].tolist(), s["lens"].tolist(), s["prefix_len"]
    shared = -(-pre // P)
    for h in range(Hkv):  # dense scores over the whole context, keys of other pages left out
        for b in range(case["B"]):
            ids = torch.cat([s["prefix"], s["table"][b, : -(-lens[b] // P)]]).long()
            k, v = (x[ids, h].reshape(-1, D).double() for x in (s["pages_k"], s["pages_v"]))
            at = torch.arange(k.shape[0], device="cuda")
            for a in range(start[b], start[b + 1], 256):
                e = min(a + 256, start[b + 1])
                taken = torch.zeros((e - a, ids.numel() + 1), dtype=torch.bool, device="cuda")
                sel = s["sel"][a:e, h].long()
                taken.scatter_(1, torch.where(sel >= 0, sel, ids.numel()), True)
                last = lens[b] - start[b + 1] + torch.arange(a, e, device="cuda")
                sees = torch.where(at < shared * P, at < pre, at - shared * P <= last[:, None])
                sees = (sees & taken[:, at // P]).repeat_interleave(r, 0)
                x = s["q"][a:e, h * r: (h + 1) * r].double().reshape(-1, D) @ k.T / D ** 0.5
                x = x.masked_fill(~sees, -float("inf"))
                z = torch.logsumexp(x, -1)
                out[a:e, h * r: (h + 1) * r] = (torch.exp(x - z[:, None]) @ v).view(e - a, r, D)
                lse[a:e, h * r: (h + 1) * r] = z.view(e - a, r)
    return {"out": out, "lse": lse}
