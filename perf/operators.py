"""Serving from a paged 8-bit cache: the four operators, their plain forms and their cases.

A cache holds `rows` requests.  Row r has `length` tokens in `held` pages of B tokens; page numbers are in
`block_table[r]`.  A complete block is held in 8 bits (e4m3 or int8) with one fp32 scale per (page, head), its mean key as
two bf16 (hi + lo); the last, partial block is held in bf16 in `tail_k`, `tail_v` (bank = block number mod 2).  `hist`
keeps the last raw keys of a row (ring by position mod 16) for the causal key convolution.
"""
import math
import random

import torch

own = False

DEV = "cuda"
QMAX = {"e4m3": 448.0, "int8": 127.0}
FLT_MIN = 2.0 ** -126


# ---------------------------------------------------------------------------------------------------------------- cases
def _lens(case):
    """Cached tokens per row before the call: over the logarithm of [len_min, len_max], the first row the longest."""
    r = random.Random(case["len_seed"])
    lo, hi = case["len_min"], case["len_max"]
    a, b = math.log(lo + 1), math.log(hi + 1)
    got = [min(hi, max(lo, int(math.exp(r.uniform(a, b))) - 1)) for _ in range(case["rows"])]
    got[0] = hi
    return got


def _news(case):
    """New tokens per row; -1 (release) for every `release`-th row of a tables case."""
    if case.get("prompts"):
        return [8192, 16384, 32768, 65536]
    r = random.Random(case["len_seed"] + 1)
    lo, hi = case["new_min"], case["new_max"]
    a, b = math.log(lo + 1), math.log(hi + 1)
    got = [min(hi, max(lo, int(math.exp(r.uniform(a, b))) - 1)) for _ in range(case["rows"])]
    got[-1] = hi
    every = case.get("release", 0)
    if every:
        got = [-1 if i % every == 1 else n for i, n in enumerate(got)]
    return got


def listed():
    base = dict(len_seed=11)
    h16 = dict(h_q=16, h_kv=16, head_dim=64, block=32, topk=32)        # the headline heads: N = 64K, B = 32, k = 32
    gqa = dict(h_q=32, h_kv=8, head_dim=128, block=64, topk=16)        # the packed GQA configuration
    return [
        # one generation step's bookkeeping: 64 requests, one token each
        dict(base, name="tables_decode_64", op="tables", rows=64, len_min=0, len_max=65536, new_min=1, new_max=1, block=32),
        # a step that admits prompts beside running and finished requests
        dict(base, name="tables_mixed_1024", op="tables", rows=1024, len_min=0, len_max=16384, new_min=0, new_max=8192,
             block=64, release=8),
        # the keys and values of one generated token for 64 requests, with the key convolution
        dict(base, name="append_decode_64_kconv4", op="append", rows=64, len_min=0, len_max=65536, new_min=1, new_max=1,
             kind="e4m3", conv=4, **h16),
        # four whole prompts of the packed GQA configuration written at once
        dict(base, name="append_prompts_120k_gqa", op="append", rows=4, len_min=0, len_max=0, new_min=0, new_max=0,
             prompts=True, kind="e4m3", conv=0, **gqa),
        # odd chunks behind odd lengths, small blocks, int8
        dict(base, name="append_ragged_int8_kconv3", op="append", rows=37, len_min=0, len_max=5003, new_min=0, new_max=701,
             kind="int8", conv=3, h_q=6, h_kv=2, head_dim=64, block=16, topk=8),
        # routing of a single request's next token: latency
        dict(base, name="route_one_64k", op="route", rows=1, len_min=65535, len_max=65535, new_min=1, new_max=1,
             kind="e4m3", conv=0, **h16),
        # routing of 64 requests of ragged lengths
        dict(base, name="route_decode_64", op="route", rows=64, len_min=1024, len_max=65535, new_min=1, new_max=1,
             kind="e4m3", conv=0, **h16),
        # routing of ragged chunks (chunked prompts, drafted tokens), grouped heads
        dict(base, name="route_chunks_gqa", op="route", rows=5, len_min=1000, len_max=65003, new_min=7, new_max=301,
             kind="e4m3", conv=0, **gqa),
        # selected attention of a single request's next token: latency
        dict(base, name="attend_one_64k", op="attend", rows=1, len_min=65535, len_max=65535, new_min=1, new_max=1,
             kind="e4m3", conv=0, select=True, **h16),
        # selected attention of 64 requests of ragged lengths: the usual serving step
        dict(base, name="attend_decode_64", op="attend", rows=64, len_min=1024, len_max=65535, new_min=1, new_max=1,
             kind="e4m3", conv=0, select=True, **h16),
        # the full-attention layers of a hybrid model, int8: the largest read
        dict(base, name="attend_all_decode_24_int8", op="attend", rows=24, len_min=4096, len_max=65535, new_min=1,
             new_max=1, kind="int8", conv=0, select=False, **gqa),
        # full attention of ragged chunks against their cache: the largest arithmetic
        dict(base, name="attend_all_chunks", op="attend", rows=3, len_min=3000, len_max=16001, new_min=200, new_max=513,
             kind="e4m3", conv=0, select=False, h_q=32, h_kv=8, head_dim=128, block=128, topk=8),
    ]


def draw(rng):
    def span(lo, hi):
        return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))

    top = {}
    for c in listed():
        w = work(c)
        for m in ("bytes", "flops"):
            top[c["op"], m] = max(top.get((c["op"], m), 0), w[m])
    while True:
        op = rng.choice(["tables", "append", "route", "attend"])
        c = dict(op=op, len_seed=rng.randrange(1 << 20), block=rng.choice([16, 32, 64, 128]))
        if op == "tables":
            c.update(rows=span(1, 1024), len_min=0, len_max=span(1, 65536), new_min=rng.choice([0, 1]),
                     new_max=span(1, 8192), release=rng.choice([0, 0, 5, 9]))
        else:
            g = rng.choice([1, 1, 2, 3, 4, 8])
            h_kv = rng.choice([1, 2, 4, 5, 8, 16])
            c.update(h_kv=h_kv, h_q=g * h_kv, head_dim=rng.choice([64, 128]), kind=rng.choice(["e4m3", "int8"]),
                     topk=span(1, 64), conv=0, len_min=0)
            if op == "append":
                c.update(rows=span(1, 256), len_max=span(1, 65536), new_min=rng.choice([0, 1]), new_max=span(1, 8192),
                         conv=rng.choice([0, 1, 2, 3, 4, 8]))
            else:
                c.update(rows=span(1, 64), len_max=span(1, 65536), new_min=1, new_max=span(1, 400))
                c["len_min"] = rng.randrange(c["len_max"])
            if op == "attend":
                c["select"] = rng.choice([True, False])
        w = work(c)
        total = sum(max(n, 0) for n in _news(c))
        if total == 0 or any(w[m] > top[op, m] for m in w):
            continue
        # what the plain forms of these spread out has to fit the card
        longest = max(_lens(c)) + max(_news(c))
        most = max(_news(c))
        if op == "route" and (max(_lens(c)) // c["block"] <= c["topk"] or c["topk"] == 1):
            continue                                            # every block is taken: nothing to route
        if op in ("route", "attend"):
            if c["rows"] * longest * c["h_kv"] * c["head_dim"] > 2 ** 31:
                continue
            if c["rows"] * most * c["h_q"] * longest > 2 ** 30 and not c.get("select"):
                continue
            if total * c["h_q"] * min(c["topk"], longest // c["block"] + 1) * c["block"] * c["head_dim"] > 2 ** 31:
                continue
            if c["rows"] * most * c["h_q"] * (longest // c["block"] + 1) > 2 ** 28:
                continue
        return c


def work(case):
    lens, news, B = _lens(case), _news(case), case["block"]
    T = sum(max(n, 0) for n in news)
    if case["op"] == "tables":
        moved = sum(-(-l // B) for l, n in zip(lens, news) if n < 0)
        taken = sum(-(-(l + n) // B) - -(-l // B) for l, n in zip(lens, news) if n > 0)
        return {"bytes": case["rows"] * 24 + 12 * T + 8 * (moved + taken), "flops": T}
    H, hq, d = case["h_kv"], case["h_q"], case["head_dim"]
    if case["op"] == "append":
        full = sum((l + n) // B - l // B for l, n in zip(lens, news) if n > 0)
        head = sum(l % B for l, n in zip(lens, news) if n > 0 and (l + n) // B > l // B)   # tail tokens read back
        left = sum(min(n, (l + n) % B + B) for l, n in zip(lens, news))                    # tail tokens written
        return {"bytes": H * d * (4 * T + 4 * head + 4 * left + full * (2 * B + 4)) + 8 * H * full,
                "flops": H * d * T * (2 * case["conv"] + 6)}
    if case["op"] == "route":
        nb = [(l + n - 1) // B for l, n in zip(lens, news)]
        return {"bytes": sum(nb) * H * d * 4 + T * hq * (2 * d + 4 * case["topk"]),
                "flops": sum(2 * n * b * hq * d for n, b in zip(news, nb))}
    if case["select"]:
        blocks = [min((l + n - 1) // B + 1, n * (hq // H) * case["topk"]) for l, n in zip(lens, news)]
        keys = sum(min(case["topk"], (l + n - 1) // B + 1) * B * n for l, n in zip(lens, news))
        return {"bytes": sum(blocks) * H * B * d * 2 + T * hq * (4 * d + 4 + 4 * case["topk"]), "flops": 4 * keys * hq * d}
    return {"bytes": sum(l + n for l, n in zip(lens, news)) * H * d * 2 + T * hq * (4 * d + 4),
            "flops": sum(4 * n * (l + (n + 1) // 2) for l, n in zip(lens, news)) * hq * d}


# --------------------------------------------------------------------------------------------------------------- inputs
def _f8(x, kind):
    if kind == "e4m3":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn)
    return torch.round(x).clamp(-127, 127).to(torch.int8)


def _pages(gen, n, H, B, d, kind, mean):
    """n pages of blocks as they come out of a model: a block's tokens share a mean, heads have their own size."""
    x8 = torch.empty((n, H, B, d), dtype=torch.float8_e4m3fn if kind == "e4m3" else torch.int8, device=DEV)
    sc = torch.empty((n, H), device=DEV)
    hi = torch.empty((n, H, d), dtype=torch.bfloat16, device=DEV)
    lo = torch.empty((n, H, d), dtype=torch.bfloat16, device=DEV)
    step = max(1, (1 << 26) // (H * B * d))
    for i in range(0, n, step):
        m = min(step, n - i)
        x = torch.randn((m, H, B, d), generator=gen, device=DEV) + mean * torch.randn((m, H, 1, d), generator=gen, device=DEV)
        x = x.bfloat16().float()
        s = (x.abs().amax((2, 3)) / QMAX[kind]).clamp_min(FLT_MIN)
        x8[i:i + m] = _f8(x / s[:, :, None, None], kind)
        c = x.mean(2)
        sc[i:i + m], hi[i:i + m] = s, c.bfloat16()
        lo[i:i + m] = (c - c.bfloat16().float()).bfloat16()
    return x8, sc, hi, lo


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 7919 + 13)
    lens, news, B, R = _lens(case), _news(case), case["block"], case["rows"]
    T = sum(max(n, 0) for n in news)
    held = [-(-l // B) for l in lens]
    after = [l + max(n, 0) for l, n in zip(lens, news)]
    total = [-(-a // B) for a in after]
    MB = max(max(total), 1) + 1
    tables = case["op"] == "tables"
    order = torch.randperm(sum(total) + 5, generator=gen, device=DEV).to(torch.int32)   # pages are handed out in no order
    P = order.numel()
    s = {"case": case, "rows": R, "T": T, "pages": P, "max_blocks": MB}
    table = torch.full((R, MB), -1, dtype=torch.int32)
    have, at = held if tables else total, 0
    host = order.cpu()
    for r in range(R):
        table[r, :have[r]] = host[at:at + have[r]]
        at += have[r]
    s["table"] = table.to(DEV)
    s["new_len"] = _i32(news)
    if tables:
        # the free pages sit anywhere in the ring: start it behind its middle
        ring0 = P // 2 + 3
        free = torch.empty(P, dtype=torch.int32, device=DEV)
        free[(torch.arange(P, device=DEV) + ring0 - at) % P] = order
        s["state"] = _i32([[l, h] for l, h in zip(lens, held)])
        s["free"], s["ring"] = free, torch.tensor([ring0, ring0 + P - at], dtype=torch.int64, device=DEV)
        if own:
            s["handle"] = _handle(s, 1, 64, B, "e4m3", 0)
            s["state_out"], s["ring_out"] = torch.empty_like(s["state"]), torch.empty_like(s["ring"])
            s["ws"] = s["handle"].alloc_workspace(T, 1)
        return s

    H, hq, d, kind = case["h_kv"], case["h_q"], case["head_dim"], case["kind"]
    s["state"] = _i32([[a, t] for a, t in zip(after, total)])
    s["free"], s["ring"] = order, torch.tensor([at, P], dtype=torch.int64, device=DEV)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + max(n, 0))
    s["cu"] = _i32(cu)
    s["token_row"] = torch.repeat_interleave(torch.arange(R, device=DEV), _i32(news).long()).to(torch.int32)
    start = _i32(lens)[s["token_row"].long()]
    s["token_pos"] = (start + torch.arange(T, device=DEV) - s["cu"][s["token_row"].long()]).to(torch.int32)
    page = s["table"][s["token_row"].long(), (s["token_pos"] // B).long()]
    s["slot"] = (page * B + s["token_pos"] % B).to(torch.int32)

    def rand16(shape, mean=0.0):
        x = torch.randn(shape, generator=gen, device=DEV)
        return (x + mean * torch.randn(shape[-2:], generator=gen, device=DEV)).bfloat16()

    s["tail_k"], s["tail_v"] = rand16((R, 2, H, B, d), 0.3), rand16((R, 2, H, B, d), 0.3)
    s["hist"] = rand16((R, 16, H, d)) if case["conv"] else None
    empty8 = dict(dtype=torch.float8_e4m3fn if kind == "e4m3" else torch.int8, device=DEV)
    if case["op"] == "append":
        s["k8"], s["v8"] = torch.zeros((P, H, B, d), **empty8), torch.zeros((P, H, B, d), **empty8)
        s["ks"], s["vs"] = torch.zeros((P, H), device=DEV), torch.zeros((P, H), device=DEV)
        s["cent"] = torch.zeros((2, P, H, d), dtype=torch.bfloat16, device=DEV)
        s["k"], s["v"] = rand16((T, H, d), 0.3), rand16((T, H, d), 0.3)
        s["w"] = torch.rand((H, d, case["conv"]), generator=gen, device=DEV) - 0.5 if case["conv"] else None
        # a chunk behind a partial block replaces what it has read of the bf16 tokens: such a step starts from a copy
        if case["len_max"] > 0 and max(news) > 1:
            s["before"] = [(s[n], s[n].clone()) for n in ("tail_k", "tail_v", "hist") if s[n] is not None]
    elif case["op"] == "route":
        # the router reads the centroids only
        s["k8"], s["v8"] = torch.zeros((P, H, B, d), **empty8), torch.zeros((P, H, B, d), **empty8)
        s["ks"], s["vs"] = torch.ones((P, H), device=DEV), torch.ones((P, H), device=DEV)
        c = torch.randn((P, H, d), generator=gen, device=DEV) * (1 / math.sqrt(B) + 0.2)
        hi = c.bfloat16()
        s["cent"] = torch.stack([hi, (c - hi.float()).bfloat16()])
        s["q"] = rand16((T, hq, d), 0.3)
    else:
        s["k8"], s["ks"], hi, lo = _pages(gen, P, H, B, d, kind, 0.3)
        s["v8"], s["vs"], _, _ = _pages(gen, P, H, B, d, kind, 0.1)
        s["cent"] = torch.stack([hi, lo])
        s["q"] = (1.5 * rand16((T, hq, d), 0.3).float()).bfloat16()
        s["sel"] = None
        if case["select"]:
            nb, k = max(total), case["topk"]
            mine = (s["token_pos"] // B).long()
            x = torch.rand((T, hq, nb), generator=gen, device=DEV)
            j = torch.arange(nb, device=DEV)
            x = torch.where(j < mine[:, None, None], x, torch.where(j == mine[:, None, None], 2.0, -1.0))
            val, idx = x.topk(min(k, nb), dim=-1)
            idx = torch.where(val < 0, nb, idx).sort(-1).values
            idx = torch.where(idx >= nb, -1, idx)
            s["sel"] = torch.nn.functional.pad(idx, (0, k - idx.shape[-1]), value=-1).to(torch.int32).contiguous()
    if own:
        s["handle"] = _handle(s, H, d, B, kind, case["conv"])
        s["plan"] = _package().CachePlan(s["cu"], s["token_row"], s["token_pos"], s["slot"])
        s["ws"] = s["handle"].alloc_workspace(T, hq)
    return s


def _package():
    from block_sparse_long_key_b200 import moba
    return moba


def _handle(s, H, d, B, kind, conv):
    """The framework's cache object over the state's own buffers (bookkeeping only for a tables case)."""
    return _package().Cache(rows=s["rows"], n_pages=s["pages"], max_blocks=s["max_blocks"], h_kv=H, head_dim=d, block_size=B,
                            kind=kind, conv_width=conv, k=s.get("k8"), v=s.get("v8"), k_scale=s.get("ks"),
                            v_scale=s.get("vs"), cent=s.get("cent"), tail_k=s.get("tail_k"), tail_v=s.get("tail_v"),
                            hist=s.get("hist"), block_table=s["table"], row_state=s["state"], free_pages=s["free"],
                            ring=s["ring"])


# ----------------------------------------------------------------------------------------------------------- plain forms
def _tables(s):
    c, B, T, P, MB = s["case"], s["case"]["block"], s["T"], s["pages"], s["max_blocks"]
    length, held = s["state"][:, 0].long(), s["state"][:, 1].long()
    n = s["new_len"].long()
    cu = torch.nn.functional.pad(n.clamp_min(0).cumsum(0), (1, 0))
    total = (length + n.clamp_min(0) + B - 1) // B
    over = total > MB
    need = torch.where(over | (n < 0), 0, (total - held).clamp_min(0))
    end = need.cumsum(0)
    ok = ~over & ((need == 0) | (end <= s["ring"][1] - s["ring"][0])) & (n >= 0)
    taken = torch.where(ok, need, 0)
    first = s["ring"][0] + end - need
    table = s["table"].clone()
    j = torch.arange(MB, device=DEV)
    fresh = (j >= held[:, None]) & (j < (held + taken)[:, None])
    at = (first[:, None] + j - held[:, None]) % P
    table = torch.where(fresh, s["free"][at.clamp_min(0)], table)
    gone = torch.where(n < 0, held, 0)
    to = s["ring"][1] + gone.cumsum(0) - gone
    free = s["free"].clone()
    leaves = j < gone[:, None]
    free[((to[:, None] + j) % P)[leaves]] = s["table"][leaves]
    after = torch.stack([torch.where(n < 0, 0, torch.where(ok, length + n, length)),
                         torch.where(n < 0, 0, held + taken)], 1).to(torch.int32)
    ring = torch.stack([s["ring"][0] + taken.sum(), s["ring"][1] + gone.sum()])
    t = torch.arange(T, device=DEV)
    row = torch.searchsorted(cu[1:], t, right=True)
    pos = torch.where(ok[row], length[row] + t - cu[row], -1)
    slot = torch.where(pos < 0, -1, table[row, (pos // B).clamp_min(0)].long() * B + pos % B)
    return {"cu": cu.to(torch.int32), "row": row.to(torch.int32), "pos": pos.to(torch.int32), "slot": slot.to(torch.int32),
            "table": table, "state": after, "ring": ring, "free": free}


def _append(s):
    c, B, W = s["case"], s["case"]["block"], s["case"]["conv"]
    row, pos, cu = s["token_row"].long(), s["token_pos"].long(), s["cu"].long()
    T, H, d = s["k"].shape
    t = torch.arange(T, device=DEV)
    rel = t - cu[row]
    k = s["k"]
    if W:
        # 64 bits: the sum is rounded to bf16 once, next to borders too
        l = torch.arange(W, device=DEV)
        fresh = s["k"][(t[:, None] - l).clamp_min(0)]
        past = s["hist"][row[:, None], (pos[:, None] - l) % 16]
        x = torch.where((l <= rel[:, None])[:, :, None, None], fresh, past).double()
        x = torch.where((l <= pos[:, None])[:, :, None, None], x, 0.0)
        z = torch.einsum("twhd,hdw->thd", x, s["w"].double())
        k = (s["k"].double() + z / (1 + torch.exp(-z))).to(torch.bfloat16)
        last = rel >= (cu[row + 1] - cu[row]) - (W - 1)
        s["hist"][row[last], pos[last] % 16] = s["k"][last]
    # one entry for each block touched: its bf16 tokens, old and new
    lead = ((pos % B == 0) | (rel == 0)).nonzero().flatten()
    run = torch.searchsorted(lead, t, right=True) - 1
    r, j = row[lead], pos[lead] // B
    old_k, old_v = s["tail_k"][r, j % 2], s["tail_v"][r, j % 2]
    old_k[run, :, pos % B] = k
    old_v[run, :, pos % B] = s["v"]
    end = s["state"][r, 0].long()
    full = (j + 1) * B <= end
    page = (s["slot"].long()[lead] // B)[full]
    for_k, for_v = old_k[full].float(), old_v[full].float()
    qmax = QMAX[c["kind"]]
    ks = (for_k.abs().amax((2, 3)) / qmax).clamp_min(FLT_MIN)
    vs = (for_v.abs().amax((2, 3)) / qmax).clamp_min(FLT_MIN)
    bits = torch.uint8
    s["k8"].view(bits)[page] = _f8(for_k / ks[:, :, None, None], c["kind"]).view(bits)
    s["v8"].view(bits)[page] = _f8(for_v / vs[:, :, None, None], c["kind"]).view(bits)
    s["ks"][page], s["vs"][page] = ks, vs
    mean = (for_k.double().sum(2) / B).float()
    hi = mean.to(torch.bfloat16)
    s["cent"][0, page], s["cent"][1, page] = hi, (mean - hi.float()).to(torch.bfloat16)
    # the last two blocks of a row stay in bf16
    keep = pos // B >= (s["state"][row, 0].long() - 1) // B - 1
    a, b, p = row[keep], (pos[keep] // B) % 2, pos[keep] % B
    s["tail_k"][a, b, :, p], s["tail_v"][a, b, :, p] = k[keep], s["v"][keep]
    return {"k8": s["k8"], "v8": s["v8"], "ks": s["ks"], "vs": s["vs"], "cent": s["cent"], "tail_k": s["tail_k"],
            "tail_v": s["tail_v"], "hist": s["hist"]}


def _by_row(s, x):
    """[T, ...] as [rows, most new tokens, ...] and the index back."""
    row = s["token_row"].long()
    rel = torch.arange(s["T"], device=DEV) - s["cu"].long()[row]
    y = torch.zeros((s["rows"], max(_news(s["case"]))) + x.shape[1:], dtype=x.dtype, device=DEV)
    y[row, rel] = x
    return y, (row, rel)


def _route(s):
    c, B, k = s["case"], s["case"]["block"], s["case"]["topk"]
    T, hq, d = s["q"].shape
    H = c["h_kv"]
    pages = s["table"][:, :s["max_blocks"] - 1].clamp_min(0).long()
    cent = s["cent"][0].double()[pages] + s["cent"][1].double()[pages]      # 64 bits: scores next to one another
    q, back = _by_row(s, s["q"].double().reshape(T, H, hq // H, d))
    x = torch.einsum("rnhgd,rjhd->rnhgj", q, cent)[back].reshape(T, hq, -1)
    mine = (s["token_pos"].long() // B)[:, None, None]
    j = torch.arange(x.shape[-1], device=DEV)
    x = torch.where(j < mine, x.nan_to_num(-math.inf, math.inf, -math.inf), -math.inf)
    top = x.sort(dim=-1, descending=True, stable=True).indices[..., :k - 1]
    top = torch.where(top < mine, top, 1 << 30)
    top = torch.cat([top, mine.expand(T, hq, 1)], -1).sort(-1).values
    top = torch.where(top < (1 << 30), top, -1)
    return torch.nn.functional.pad(top, (0, k - top.shape[-1]), value=-1).to(torch.int32)


def _blocks(s, x8, scale, tail, row, j, head):
    """The fp32 tokens of blocks j of rows `row` (index tensors of one shape): from the page, or the tail where it is partial."""
    page = s["table"][row, j].long().clamp_min(0)
    B = s["case"]["block"]
    if s["case"]["kind"] == "e4m3":
        x = x8.view(torch.uint8)[page, head].view(torch.float8_e4m3fn).float()
    else:
        x = x8[page, head].float()
    x = x * scale[page, head][..., None, None]
    full = ((j + 1) * B <= s["state"][row, 0])[..., None, None]
    return torch.where(full, x, tail[row, j % 2, head].float())


def _attend(s):
    c, B = s["case"], s["case"]["block"]
    T, hq, d = s["q"].shape
    H, G = c["h_kv"], hq // c["h_kv"]
    off = torch.arange(B, device=DEV)
    if s["sel"] is not None:
        row = s["token_row"].long()[:, None, None].expand_as(s["sel"])
        j = s["sel"].long().clamp_min(0)
        head = (torch.arange(hq, device=DEV) // G)[None, :, None].expand_as(j)
        seen = (s["sel"] >= 0)[..., None] & (j[..., None] * B + off <= s["token_pos"][:, None, None, None])
        k = _blocks(s, s["k8"], s["ks"], s["tail_k"], row, j, head).flatten(2, 3)
        x = torch.einsum("thd,thld->thl", s["q"].float(), k) / math.sqrt(d)
        del k
        x = torch.where(seen.flatten(2), x, -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m)
        v = torch.where(seen.flatten(2)[..., None], _blocks(s, s["v8"], s["vs"], s["tail_v"], row, j, head).flatten(2, 3), 0)
        l = p.sum(-1, keepdim=True)
        o = torch.einsum("thl,thld->thd", p, v) / l
        return o.to(torch.bfloat16), (m + torch.log(l))[..., 0]
    nb = s["max_blocks"] - 1
    row = torch.arange(s["rows"], device=DEV)[:, None, None].expand(-1, H, nb)
    j = torch.arange(nb, device=DEV)[None, None].expand_as(row)
    head = torch.arange(H, device=DEV)[None, :, None].expand_as(row)
    q, back = _by_row(s, s["q"].float().reshape(T, H, G, d))
    pos, _ = _by_row(s, s["token_pos"].long())
    k = _blocks(s, s["k8"], s["ks"], s["tail_k"], row, j, head).flatten(2, 3)
    x = torch.einsum("rnhgd,rhld->rnhgl", q, k) / math.sqrt(d)
    del k
    seen = torch.arange(nb * B, device=DEV) <= pos[:, :, None, None, None]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    del x
    l = p.sum(-1, keepdim=True)
    v = _blocks(s, s["v8"], s["vs"], s["tail_v"], row, j, head).flatten(2, 3)
    live = (torch.arange(nb * B, device=DEV) < s["state"][:, :1])[:, None, :, None]
    o = torch.einsum("rnhgl,rhld->rnhgd", p, torch.where(live, v, 0)) / l
    return o[back].reshape(T, hq, d).to(torch.bfloat16), (m + torch.log(l))[back].reshape(T, hq)


def run(s):
    op = s["case"]["op"]
    if s.get("before"):
        torch._foreach_copy_([x for x, _ in s["before"]], [y for _, y in s["before"]])
    if own:
        moba = _package()
        h = s["handle"]
        if op == "tables":
            p = moba.cache_tables(h, s["new_len"], s["T"], row_state_out=s["state_out"], ring_out=s["ring_out"],
                                  workspace=s["ws"])
            return {"cu": p.cu_new, "row": p.token_row, "pos": p.token_pos, "slot": p.slot_map, "table": s["table"],
                    "state": s["state_out"], "ring": s["ring_out"], "free": s["free"]}
        if op == "append":
            moba.cache_append(h, s["plan"], s["k"], s["v"], conv_w=s["w"], workspace=s["ws"])
            return {"k8": s["k8"], "v8": s["v8"], "ks": s["ks"], "vs": s["vs"], "cent": s["cent"],
                    "tail_k": s["tail_k"], "tail_v": s["tail_v"], "hist": s["hist"]}
        if op == "route":
            return moba.cache_route(h, s["plan"], s["q"], s["case"]["topk"], workspace=s["ws"])
        return moba.cache_attention(h, s["plan"], s["q"], sel_idx=s["sel"], workspace=s["ws"])
    return {"tables": _tables, "append": _append, "route": _route, "attend": _attend}[op](s)


# --------------------------------------------------------------------------------------------------- 64-bit definition
def exact(case, seed):
    """By request and in float64, from the definition; whole numbers have none."""
    if case["op"] in ("tables", "route"):
        return None
    s = prepare(case, seed)
    lens, news, B, H, d = _lens(case), _news(case), case["block"], case["h_kv"], case["head_dim"]
    f = torch.float64
    starts = s["cu"].tolist()
    if case["op"] == "append":
        W = case["conv"]
        k8 = s["k8"].to(f) if case["kind"] == "e4m3" else None
        v8 = s["v8"].to(f) if case["kind"] == "e4m3" else None
        ks, vs, cent = s["ks"].to(f), s["vs"].to(f), s["cent"].to(f)
        tk, tv = s["tail_k"].to(f), s["tail_v"].to(f)
        hist = s["hist"].to(f) if W else None
        table = s["table"].cpu()
        for r, (L, n) in enumerate(zip(lens, news)):
            if n <= 0:
                continue
            raw = s["k"][starts[r]:starts[r] + n].to(f)
            val = s["v"][starts[r]:starts[r] + n].to(f)
            key = raw
            if W:
                before = [s["hist"][r, p % 16].to(f) if p >= 0 else torch.zeros((H, d), dtype=f, device=DEV)
                          for p in range(L - W + 1, L)]
                line = torch.cat([torch.stack(before), raw]) if before else raw
                z = sum(line[W - 1 - l:W - 1 - l + n] * s["w"][:, :, l].to(f) for l in range(W))
                key = raw + z * torch.sigmoid(z)
                for p in range(max(L, L + n - W + 1), L + n):
                    hist[r, p % 16] = raw[p - L]
            rounded = key.to(torch.bfloat16).to(f)      # what the cache keeps of a key
            first, last = L // B, (L + n - 1) // B
            for tail, new, x8, sc, is_key in ((tk, rounded, k8, ks, True), (tv, val, v8, vs, False)):
                old = L - first * B
                line = torch.cat([tail[r, first % 2, :, :old].transpose(0, 1), new])
                done = (L + n) // B - first
                if done > 0:
                    blk = line[:done * B].reshape(done, B, H, d).transpose(1, 2)
                    pg = table[r, first:first + done].long().to(DEV)
                    scale = (blk.abs().amax((2, 3)) / QMAX[case["kind"]]).clamp_min(FLT_MIN)
                    sc[pg] = scale
                    if x8 is not None:
                        x8[pg] = blk / scale[:, :, None, None]
                    if is_key:
                        mean = blk.mean(2)
                        hi = mean.to(torch.bfloat16)
                        cent[0, pg], cent[1, pg] = hi.to(f), mean - hi.to(f)
                for b in range(max(first, last - 1), last + 1):
                    lo, up = max(L, b * B), min(L + n, (b + 1) * B)
                    tail[r, b % 2, :, lo - b * B:up - b * B] = (key if is_key else val)[lo - L:up - L].transpose(0, 1)
        return {"k8": k8, "v8": v8, "ks": ks, "vs": vs, "cent": cent, "tail_k": tk, "tail_v": tv, "hist": hist}
    hq = case["h_q"]
    G = hq // H
    out = torch.empty((s["T"], hq, d), dtype=f, device=DEV)
    lse = torch.empty((s["T"], hq), dtype=f, device=DEV)
    for r, (L, n) in enumerate(zip(lens, news)):
        full, left = (L + n) // B, (L + n) % B
        pg = s["table"][r, :full].long()
        for h in range(H):
            kk = (s["k8"][:, h].view(torch.uint8)[pg].view(s["k8"].dtype).to(f) * s["ks"][pg, h].to(f)[:, None, None]).reshape(-1, d)
            vv = (s["v8"][:, h].view(torch.uint8)[pg].view(s["v8"].dtype).to(f) * s["vs"][pg, h].to(f)[:, None, None]).reshape(-1, d)
            kk = torch.cat([kk, s["tail_k"][r, full % 2, h, :left].to(f)])
            vv = torch.cat([vv, s["tail_v"][r, full % 2, h, :left].to(f)])
            for g in range(G):
                a, b = starts[r], starts[r] + n
                sc = s["q"][a:b, h * G + g].to(f) @ kk.T / math.sqrt(d)
                at = torch.arange(L + n, device=DEV)
                hide = at[None] > s["token_pos"][a:b, None]
                if s["sel"] is not None:
                    got = torch.zeros((n, full + 2), dtype=torch.bool, device=DEV)
                    j = s["sel"][a:b, h * G + g].long()
                    got.scatter_(1, torch.where(j < 0, full + 1, j), True)
                    hide |= ~got[:, at // B]
                sc.masked_fill_(hide, -math.inf)
                lse[a:b, h * G + g] = torch.logsumexp(sc, -1)
                out[a:b, h * G + g] = torch.softmax(sc, -1) @ vv
    return out, lse
