"""The paged 8-bit cache: tables, append, routing and attention, alone and as a serving run, against a plain 64-bit
cache (cache_ref.py).  Bookkeeping, 8-bit codes, scales, centroids, tails and selections are compared bit for bit."""
import ctypes

import pytest
import torch

import cache_ref as cr
from block_sparse_long_key_b200 import build, moba

gpu = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ host checks (CPU)
@pytest.fixture(scope="module")
def L():
    build.build()
    return moba.lib()


FAKE = 1 << 20  # a 16- and 256-byte aligned address that the checks never follow


def _struct(**kw):
    base = dict(rows=4, n_pages=64, max_blocks=16, h_kv=2, head_dim=64, block_size=32, kind=0, conv_width=0)
    base.update({n: FAKE for n in ("k", "v", "k_scale", "v_scale", "cent", "tail_k", "tail_v", "block_table",
                                   "row_state", "free_pages", "ring")})
    base.update(kw)
    return moba.CacheStruct(**base)


def _plan(**kw):
    base = dict(total_new=4, cu_new=FAKE, token_row=FAKE, token_pos=FAKE, slot_map=FAKE)
    base.update(kw)
    return moba.PlanStruct(**base)


@pytest.mark.parametrize("bad", [dict(head_dim=96), dict(block_size=48), dict(kind=2), dict(conv_width=9),
                                 dict(conv_width=-1), dict(rows=0), dict(n_pages=0), dict(max_blocks=0), dict(h_kv=0),
                                 dict(n_pages=1 << 26), dict(max_blocks=1 << 26)], ids=str)
def test_bad_cache_sizes_are_refused(L, bad):
    c, p = _struct(**bad), _plan()
    ref, pr = ctypes.byref(c), ctypes.byref(p)
    assert L.moba_cache_workspace_size(ref, 4, 2) == 0
    assert L.moba_cache_reset(ref, None) == moba.MOBA_EINVAL
    assert L.moba_cache_tables(ref, FAKE, None, None, pr, FAKE, 1 << 30, None) == moba.MOBA_EINVAL
    assert L.moba_cache_append(ref, pr, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == moba.MOBA_EINVAL
    assert L.moba_cache_route(ref, pr, FAKE, 2, 4, FAKE, FAKE, 1 << 30, None) == moba.MOBA_EINVAL
    assert L.moba_cache_attention(ref, pr, FAKE, 2, None, 1, FAKE, FAKE, FAKE, 1 << 30, None) == moba.MOBA_EINVAL


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "cent", "tail_k", "tail_v", "block_table",
                                  "row_state"])
def test_missing_and_misaligned_buffers_are_refused(L, name):
    p = _plan()
    for value, rc in ((None, moba.MOBA_EINVAL), (FAKE + 8, moba.MOBA_EALIGN)):
        c = _struct(**{name: value})
        ref, pr = ctypes.byref(c), ctypes.byref(p)
        assert L.moba_cache_reset(ref, None) == rc
        assert L.moba_cache_append(ref, pr, FAKE, FAKE, None, FAKE, 1 << 30, None) == rc
        assert L.moba_cache_attention(ref, pr, FAKE, 2, None, 1, FAKE, FAKE, FAKE, 1 << 30, None) == rc


def test_call_arguments_are_refused(L):
    c, p = _struct(), _plan()
    ref, pr = ctypes.byref(c), ctypes.byref(p)
    E, A, W = moba.MOBA_EINVAL, moba.MOBA_EALIGN, moba.MOBA_EWORKSPACE
    big = 1 << 40
    assert L.moba_cache_tables(ref, None, None, None, pr, FAKE, big, None) == E
    assert L.moba_cache_tables(ref, FAKE, FAKE + 4, None, pr, FAKE, big, None) == A
    assert L.moba_cache_tables(ref, FAKE, None, None, pr, FAKE, 256, None) == W
    assert L.moba_cache_tables(ref, FAKE, None, None, pr, FAKE + 128, big, None) == A
    assert L.moba_cache_tables(ref, FAKE, None, None, None, FAKE, big, None) == E
    for field in ("cu_new", "token_row", "token_pos", "slot_map"):
        q = _plan(**{field: None})
        assert L.moba_cache_tables(ref, FAKE, None, None, ctypes.byref(q), FAKE, big, None) == E
        assert L.moba_cache_route(ref, ctypes.byref(q), FAKE, 2, 4, FAKE, FAKE, big, None) == E
    neg = _plan(total_new=-1)
    assert L.moba_cache_append(ref, ctypes.byref(neg), FAKE, FAKE, None, FAKE, big, None) == E
    assert L.moba_cache_append(ref, pr, None, FAKE, None, FAKE, big, None) == E
    conv = _struct(conv_width=4, hist=FAKE)
    assert L.moba_cache_append(ctypes.byref(conv), pr, FAKE, FAKE, None, FAKE, big, None) == E
    nohist = _struct(conv_width=4)
    assert L.moba_cache_append(ctypes.byref(nohist), pr, FAKE, FAKE, FAKE, FAKE, big, None) == E
    for hq, topk in ((3, 4), (0, 4), (2, 0), (2, 65)):
        assert L.moba_cache_route(ref, pr, FAKE, hq, topk, FAKE, FAKE, big, None) == E
        assert L.moba_cache_attention(ref, pr, FAKE, hq, FAKE, topk, FAKE, FAKE, FAKE, big, None) == E
    assert L.moba_cache_route(ref, pr, FAKE, 2, 4, FAKE + 4, FAKE, big, None) == A
    assert L.moba_cache_route(ref, pr, FAKE, 2, 4, FAKE, FAKE, 255, None) == W
    assert L.moba_cache_attention(ref, pr, FAKE, 2, None, 1, None, FAKE, FAKE, big, None) == E
    huge = _plan(total_new=1 << 24)
    assert L.moba_cache_attention(ref, ctypes.byref(huge), FAKE, 2, None, 1, FAKE, FAKE, FAKE, big, None) == E
    assert L.moba_cache_workspace_size(ref, 1 << 24, 2) == 0
    none = _plan(total_new=0, token_row=None, token_pos=None, slot_map=None)  # nothing to do: nothing launched
    assert L.moba_cache_append(ref, ctypes.byref(none), None, None, None, None, 0, None) == moba.MOBA_OK
    assert L.moba_cache_route(ref, ctypes.byref(none), None, 2, 4, None, None, 0, None) == moba.MOBA_OK
    assert L.moba_cache_attention(ref, ctypes.byref(none), None, 2, None, 1, None, None, None, 0, None) == moba.MOBA_OK


def test_binding_refuses_host_tensors_and_kinds():
    with pytest.raises(TypeError):
        moba.Cache(rows=1, n_pages=4, max_blocks=4, h_kv=1, head_dim=64, block_size=16,
                   block_table=torch.zeros((1, 4), dtype=torch.int32))
    with pytest.raises(ValueError):
        moba.Cache(rows=1, n_pages=4, max_blocks=4, h_kv=1, head_dim=64, block_size=16, kind="e5m2")
    with pytest.raises(ValueError):
        moba.Cache(rows=1, n_pages=4, max_blocks=4, h_kv=1, head_dim=64, block_size=16)


# ---------------------------------------------------------------------------------------------------- serving runs (GPU)
class Run:
    """A cache on the GPU and the plain one beside it."""

    def __init__(self, rows, n_pages, max_blocks, h_q, h_kv, d, B, kind, W, topk, seed=0, scale=1.0):
        self.c = moba.alloc_cache(rows, n_pages, max_blocks, h_kv, d, B, kind=kind, conv_width=W)
        # what was never written is never read: NaN scales and pages of NaN codes
        self.c.k.view(torch.uint8).fill_(0x7F), self.c.v.view(torch.uint8).fill_(0x7F)
        for x in (self.c.k_scale, self.c.v_scale, self.c.cent, self.c.tail_k, self.c.tail_v):
            x.fill_(float("nan"))
        self.ref = cr.RefCache(rows, n_pages, max_blocks, h_kv, d, B, kind, W)
        self.hq, self.topk, self.scale, self.check = h_q, topk, scale, True
        self.gen = torch.Generator().manual_seed(seed)
        self.w = torch.rand((h_kv, d, W), generator=self.gen) - 0.5 if W else None

    def rand(self, *shape):
        return (self.scale * torch.randn(shape, generator=self.gen)).to(torch.bfloat16)

    def tables(self, new_len, pad=0, total=None):
        T = (sum(max(n, 0) for n in new_len) if total is None else total) + pad
        ws = self.c.alloc_workspace(T, self.hq)
        plan = moba.cache_tables(self.c, torch.tensor(new_len, dtype=torch.int32, device="cuda"), T, workspace=ws)
        status = moba.check_status(ws)
        want = self.ref.tables(new_len, T)
        for got, exp, name in zip(plan, want, ("cu", "row", "pos", "slot")):
            assert got.tolist() == exp, name
        self.check_state()
        return plan, want, status

    def check_state(self):
        r = self.ref
        assert self.c.row_state.tolist() == [[a, len(b)] for a, b in zip(r.length, r.pages)]
        table = self.c.block_table.tolist()
        for i in range(r.rows):
            assert table[i][:len(r.pages[i])] == r.pages[i]
        head, tail = self.c.ring.tolist()
        ring = self.c.free_pages.tolist()
        assert [ring[i % r.n_pages] for i in range(head, tail)] == list(r.free)

    def append(self, plan, want, k=None, v=None):
        T = plan.token_row.shape[0]
        r = self.ref
        k = self.rand(T, r.h, r.d) if k is None else k
        v = self.rand(T, r.h, r.d) if v is None else v
        ws = self.c.alloc_workspace(T, self.hq)
        moba.cache_append(self.c, plan, k.cuda(), v.cuda(), conv_w=None if self.w is None else self.w.cuda(),
                          workspace=ws)
        status = moba.check_status(ws)
        r.append(want[0], want[4], k, v, self.w)
        if self.check:
            self.check_store()
        return status

    def check_store(self, rows=None):
        r = self.ref
        k8, v8 = self.c.k.view(torch.uint8).cpu(), self.c.v.view(torch.uint8).cpu()
        ks, vs, cent = self.c.k_scale.cpu(), self.c.v_scale.cpu(), self.c.cent.cpu()
        tk, tv = self.c.tail_k.cpu(), self.c.tail_v.cpu()
        for i in range(r.rows) if rows is None else rows:
            for j in range(r.length[i] // r.B):
                pg = r.pages[i][j]
                for x, codes, scales, what in ((r.key, k8, ks, "k"), (r.val, v8, vs, "v")):
                    c, s = r.block(x, i, j)
                    assert torch.equal(scales[pg], s), (what, i, j)
                    a, b = codes[pg], c.view(torch.uint8)
                    if r.kind == "e4m3":   # +0 and -0 are one value
                        a, b = torch.where(a == 128, 0, a), torch.where(b == 128, 0, b)
                    assert torch.equal(a, b), (what, i, j)
                # sums of up to 8 tokens are rounded to 32 bits (2^-24 of their magnitudes each), then hi + lo keep
                # the mean to 2^-17
                hi, lo = r.centroid(i, j)
                x = r.key[i][j * r.B:(j + 1) * r.B].double()
                off = (cent[0, pg].double() + cent[1, pg].double() - x.mean(0)).abs()
                assert (off <= 2.0 ** -17 * (1 + 2.0 ** -6) * x.mean(0).abs() + 8 * 2.0 ** -24 * x.abs().mean(0)).all(), (i, j)
                assert (cent[0, pg] == hi).float().mean() > 0.99, (i, j)
                r.cents[pg] = cent[0, pg].double() + cent[1, pg].double()   # what routing reads
            left, j = r.length[i] % r.B, r.length[i] // r.B
            if left:
                assert torch.equal(tk[i, j % 2, :, :left].transpose(0, 1), r.key[i][j * r.B:]), i
                assert torch.equal(tv[i, j % 2, :, :left].transpose(0, 1), r.val[i][j * r.B:]), i

    def queries(self, plan, want, q=None, dense=True):
        T = plan.token_row.shape[0]
        r = self.ref
        q = self.rand(T, self.hq, r.d) if q is None else q
        ws = self.c.alloc_workspace(T, self.hq)
        sel0 = torch.full((T, self.hq, self.topk), -7, dtype=torch.int32, device="cuda")
        sel = moba.cache_route(self.c, plan, q.cuda(), self.topk, workspace=ws, sel_idx=sel0)
        assert moba.check_status(ws) == 0
        row, pos = want[1], want[2]
        exp = r.route(row, pos, q, self.topk)
        real = torch.tensor([x >= 0 for x in row])
        assert torch.equal(sel.cpu()[real], exp[real])
        assert (sel.cpu()[~real] == -7).all()          # padding rows stay as they were
        for s_gpu, s_ref in ((sel, exp), (None, None))[:2 if dense else 1]:
            out = torch.full((T, self.hq, r.d), 7.0, dtype=torch.bfloat16, device="cuda")
            lse = torch.full((T, self.hq), 7.0, device="cuda")
            ws.random_(0, 255)
            moba.cache_attention(self.c, plan, q.cuda(), sel_idx=s_gpu, workspace=ws, out=out, lse=lse)
            assert moba.check_status(ws) == 0
            ref = r.attend(row, pos, q, s_ref)
            cr.check_attention(out.cpu()[real], lse.cpu()[real], [x[real] for x in ref], r.d,
                               "all" if s_ref is None else "selected")
            assert (out.cpu()[~real] == 7).all() and (lse.cpu()[~real] == 7).all()
        return sel

    def step(self, new_len, pad=0, dense=True):
        plan, want, st = self.tables(new_len, pad)
        assert st == 0
        if plan.token_row.shape[0]:
            assert self.append(plan, want) == 0
            self.queries(plan, want, dense=dense)


# (h_q, h_kv, d, B, kind, conv width, topk)
SHAPES = [
    (2, 2, 64, 32, "e4m3", 4, 4),
    (4, 1, 64, 16, "int8", 3, 3),
    (6, 2, 128, 64, "e4m3", 0, 2),
    (8, 4, 128, 16, "int8", 8, 64),
    (1, 1, 64, 128, "int8", 2, 1),
    (5, 5, 128, 128, "e4m3", 1, 3),
    (24, 1, 64, 32, "e4m3", 0, 5),
]


def _ids(s):
    return "h%dx%d_d%d_B%d_%s_w%d_k%d" % s


@gpu
@pytest.mark.parametrize("shape", SHAPES, ids=_ids)
def test_serving_run(shape):
    """Prompts, single tokens, chunks across blocks, idle rows, a finished row and its successor, padding."""
    hq, h, d, B, kind, W, topk = shape
    r = Run(5, 400 // B + 40, 600 // B + 6, hq, h, d, B, kind, W, topk, seed=B + d)
    r.step([B * 3 + 5, 1, 0, B, 2 * B - 1], pad=3)
    r.step([1, 1, 1, 1, 1])
    r.step([1, 0, 2, 0, 1], pad=2)
    r.step([3, B, -1, 2 * B + 3, 7])
    r.step([0, 0, B + 1, 0, 0])
    r.step([4 * B + 2, 9, 17, 2, 1], pad=1)
    for _ in range(3):
        r.step([1, 1, 1, 1, 1])


@gpu
@pytest.mark.parametrize("hq,h,d,B,kind,n,scale", [
    (4, 1, 128, 64, "e4m3", (300, 129, 1), 1.0),      # several key tiles, rows ending inside one
    (3, 1, 64, 16, "int8", (257, 40, 128), 4.0),      # sharp softmax: references move
    (16, 2, 64, 128, "e4m3", (127, 128, 2), 0.05),    # whole and all-but-whole key tiles, flat softmax
    (2, 2, 128, 32, "int8", (513, 64, 64), 30.0),     # one key takes all
], ids=str)
def test_chunks_of_many_tokens(hq, h, d, B, kind, n, scale):
    r = Run(2, 1400 // B + 4, 1100 // B + 8, hq, h, d, B, kind, 0, 4, seed=B + hq, scale=scale)
    for a in n:
        r.step([a, a // 2 + 1])


# A request goes to tiles of 128 query rows from 64 (d = 128) or 96 (d = 64) on, another of the same step to small ones.
MIXED = [
    # long rows are cut into splits; lists of new tokens around the limit
    ((8, 2, 128, 64, "e4m3"), [2500, 700, 0, 1300, 64, 1], [[1, 17, 16, 15, 1, 0], [1, 1, 1, 130, 1, 1], [33, 0, 0, 0, 0, 0]]),
    ((2, 2, 64, 32, "int8"), [2600, 900, 31, 0], [[1, 97, 96, 95], [0, 2, 193, 1], [100, 100, 1, 128]]),
    ((24, 1, 64, 16, "e4m3"), [1400, 40, 3, 800, 0], [[3, 4, 5, 1, 0], [1, 1, 1, 1, 1], [4, 0, 0, 4, 2]]),
    ((48, 1, 128, 128, "int8"), [1300, 129, 0], [[1, 1, 1], [2, 1, 0], [0, 3, 9]]),
    ((4, 1, 128, 32, "e4m3"), [3000], [[15], [16], [50]]),
    ((128, 1, 128, 64, "e4m3"), [900, 40, 5], [[1, 1, 1], [2, 0, 1], [1, 3, 0]]),     # one token is past the limit
    ((96, 1, 64, 32, "int8"), [40, 700], [[1, 1], [0, 2], [1, 0]]),
    ((1, 1, 128, 16, "int8"), [1100] + [20] * 40, [[1] * 41, [0] * 20 + [64] + [1] * 20, [2] * 40 + [70]]),
]


@gpu
@pytest.mark.parametrize("shape,held,steps", MIXED, ids=lambda x: str(x) if isinstance(x, tuple) else None)
def test_steps_of_long_chunks_and_single_tokens(shape, held, steps):
    hq, h, d, B, kind = shape
    r = Run(len(held), sum(n // B + 20 for n in held), max(held) // B + 24, hq, h, d, B, kind, 0, 3, seed=B + hq)
    plan, want, _ = r.tables(held)
    assert r.append(plan, want) == 0
    for i, new in enumerate(steps):
        r.step(new, pad=(0, 3, 40)[i])


def _route_alone(cent, q, own_tokens, B, topk, max_blocks=None, T_pad=0):
    """cache_route on centroids given as float64 [blocks, h, d] (split into hi + lo here), one row whose last token is
    the query's; returns sel [1, h_q, topk] and the centroids as held."""
    nb, h, d = cent.shape
    c = moba.alloc_cache(1, nb + 2, max_blocks or nb + 2, h, d, B)
    hi = cent.float().to(torch.bfloat16)
    lo = (cent.float() - hi.float()).to(torch.bfloat16)
    c.cent[0, :nb], c.cent[1, :nb] = hi.cuda(), lo.cuda()
    perm = torch.randperm(nb + 2, generator=torch.Generator().manual_seed(3))
    c.cent[:] = torch.cat([c.cent[:, :nb], torch.zeros((2, 2, h, d), device="cuda", dtype=torch.bfloat16)], 1)[:, torch.argsort(perm)]
    c.block_table[0, :nb + 1] = perm[:nb + 1].to(torch.int32).cuda()
    c.row_state[0, 0], c.row_state[0, 1] = own_tokens + 1, own_tokens // B + 1
    T = q.shape[0]
    i32 = dict(dtype=torch.int32, device="cuda")
    plan = moba.CachePlan(torch.tensor([0, T], **i32), torch.zeros(T, **i32), torch.full((T,), own_tokens, **i32),
                          torch.zeros(T, **i32))
    ws = c.alloc_workspace(T, q.shape[1])
    sel = moba.cache_route(c, plan, q.cuda(), topk, workspace=ws)
    assert moba.check_status(ws) == 0
    return sel.cpu(), hi.double() + lo.double()


def _route_exact(held, q, own, topk):
    h = held.shape[1]
    g = q.shape[1] // h
    sel = torch.full(q.shape[:2] + (topk,), -1, dtype=torch.int32)
    for t in range(q.shape[0]):
        for i in range(q.shape[1]):
            x = (held[:own, i // g] * q[t, i].double()).sum(-1)
            x = torch.where(torch.isnan(x), float("-inf"), x)
            got = sorted(torch.sort(x, descending=True, stable=True).indices[:topk - 1].tolist()) + [own]
            sel[t, i, :len(got)] = torch.tensor(got, dtype=torch.int32)
    return sel


@gpu
@pytest.mark.parametrize("topk", [2, 17, 64])
@pytest.mark.parametrize("what", ["random", "all_equal", "few_values", "lo_decides", "huge", "inf_query", "nan_query",
                                  "zero_query", "tiny"])
def test_routing_ties_and_extremes(what, topk):
    g = torch.Generator().manual_seed(topk)
    nb, h, d, B, T = 1500, 2, 64, 16, 3
    cent = torch.randn((nb, h, d), generator=g).double()
    q = torch.randn((T, 4, d), generator=g).to(torch.bfloat16)
    if what == "all_equal":                     # every block a candidate: the list overflows, ties go to lower blocks
        cent[:] = cent[:1]
    elif what == "few_values":                  # small integers: sums are exact, many ties
        cent, q = torch.randint(-1, 2, (nb, h, d), generator=g).double(), torch.randint(-1, 2, (T, 4, d), generator=g).to(torch.bfloat16)
    elif what == "lo_decides":                  # blocks that differ below bf16 only
        cent = cent[:1] * (1 + torch.randint(-60, 60, (nb, 1, 1), generator=g).double() * 2.0 ** -16)
    elif what == "huge":                        # 32-bit sums overflow, 64-bit ones do not
        cent, q = cent * 1e25, (q.float() * 1e20).to(torch.bfloat16)
    elif what == "inf_query":
        q[1, 0, 3] = float("inf")
    elif what == "nan_query":
        q[1, 0, 3] = float("nan")
    elif what == "zero_query":
        q[:] = 0
    elif what == "tiny":                        # products below the normal range of 32 bits
        cent, q = cent * 1e-25, (q.float() * 1e-20).to(torch.bfloat16)
    own = nb - 1
    sel, held = _route_alone(cent, q, own * B + 5, B, topk)
    assert torch.equal(sel, _route_exact(held, q, own, topk))


@gpu
@pytest.mark.parametrize("own", [0, 1, 3, 4, 5, 127, 128, 129, 255, 256, 257, 600])
def test_routing_around_the_sizes_of_its_steps(own):
    g = torch.Generator().manual_seed(own)
    cent = torch.randn((own + 1, 1, 128), generator=g).double()
    q = torch.randn((2, 3, 128), generator=g).to(torch.bfloat16)
    for topk in (1, 5, 64):
        sel, held = _route_alone(cent, q, own * 32, 32, topk, max_blocks=own + 7)
        assert torch.equal(sel, _route_exact(held, q, own, topk)), topk


@gpu
def test_routing_in_slabs():
    """More screen scores than the workspace holds at a time: the tokens go through in parts."""
    g = torch.Generator().manual_seed(1)
    cent = torch.randn((40, 1, 64), generator=g).double()
    T, hq = 700, 24
    q = torch.randn((T, hq, 64), generator=g).to(torch.bfloat16)
    sel, held = _route_alone(cent, q, 39 * 16, 16, 6, max_blocks=9000)
    x = torch.einsum("thd,jd->thj", q.double(), held[:39, 0])
    want = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :5].sort(-1).values
    assert torch.equal(sel[..., :5].long(), want) and (sel[..., 5] == 39).all()


# --------------------------------------------------------------------------------------------------------- bookkeeping
def _tables_only(rows, n_pages, max_blocks, B):
    i32 = dict(dtype=torch.int32, device="cuda")
    return moba.Cache(rows=rows, n_pages=n_pages, max_blocks=max_blocks, h_kv=1, head_dim=64, block_size=B,
                      block_table=torch.full((rows, max_blocks), -1, **i32), row_state=torch.zeros((rows, 2), **i32),
                      free_pages=torch.arange(n_pages, **i32), ring=torch.tensor([0, n_pages], device="cuda"))


def _check_tables(c, ref, new_len, T, **kw):
    ws = c.alloc_workspace(0)
    plan = moba.cache_tables(c, torch.tensor(new_len, dtype=torch.int32, device="cuda"), T, workspace=ws, **kw)
    status = moba.check_status(ws)
    want = ref.tables(new_len, T)
    for got, exp, name in zip(plan, want, ("cu", "row", "pos", "slot")):
        assert got.tolist() == exp, name
    return status, want


@gpu
@pytest.mark.parametrize("rows,scale", [(7, 40), (1500, 12), (300, 300)])
def test_tables_over_many_steps(rows, scale):
    """Pages wander through the ring: growth, release, refusals, rows of nothing; one CTA's worth of rows and more, steps
    that end in the first launch and that need the second."""
    B, g = 16, torch.Generator().manual_seed(rows)
    n_pages = rows * scale // B // 2 + 9
    c, ref = _tables_only(rows, n_pages, 3 * scale // B + 4, B), cr.RefCache(rows, n_pages, 3 * scale // B + 4, 1, 64, B, "e4m3", 0)
    seen = 0
    for step in range(12):
        new = torch.randint(0, scale, (rows,), generator=g)
        new[torch.rand(rows, generator=g) < 0.3] = 0
        new[torch.rand(rows, generator=g) < 0.2] = -1
        new = new.tolist()
        T = sum(max(n, 0) for n in new) + (step % 3)
        status, want = _check_tables(c, ref, new, T)
        assert bool(status & moba.STATUS_NO_PAGES) == bool(want[4])
        assert status & ~moba.STATUS_NO_PAGES == 0
        seen |= bool(want[4])
        head, tail = c.ring.tolist()
        ring = c.free_pages.tolist()
        assert [ring[i % n_pages] for i in range(head, tail)] == list(ref.free)
        assert c.row_state.tolist() == [[a, len(b)] for a, b in zip(ref.length, ref.pages)]
    assert seen and head > n_pages        # refusals happened, and the ring went round


@gpu
def test_tables_refuse_more_tokens_and_blocks_than_there_is_room_for():
    c, ref = _tables_only(4, 100, 3, 16), cr.RefCache(4, 100, 3, 1, 64, 16, "e4m3", 0)
    status, want = _check_tables(c, ref, [48, 49, 5, 5], 107)
    assert status == moba.STATUS_NO_PAGES and want[4] == [1]
    status, want = _check_tables(c, ref, [0, 3, 40, 9], 40)          # row 2 runs past the token arrays, row 3 begins there
    assert status == moba.STATUS_BAD_SEQLENS and want[4] == [2, 3]
    assert _check_tables(c, ref, [0, 0, 0, 0], 0)[0] == 0            # nothing at all
    assert _check_tables(c, ref, [-1, -1, -1, -1], 3)[0] == 0
    assert c.row_state.tolist() == [[0, 0]] * 4


@gpu
def test_tables_out_of_place_plan_the_same_step_again():
    B = 32
    c, ref = _tables_only(5, 40, 9, B), cr.RefCache(5, 40, 9, 1, 64, B, "e4m3", 0)
    _check_tables(c, ref, [70, 3, 0, 31, 33], 137)
    state, ring = c.row_state.clone(), c.ring.clone()
    so, ro = torch.empty_like(state), torch.empty_like(ring)
    new = [2, 40, 1, -1, 31]
    ws = c.alloc_workspace(0)
    first = None
    for _ in range(3):
        p = moba.cache_tables(c, torch.tensor(new, dtype=torch.int32, device="cuda"), 74, row_state_out=so, ring_out=ro, workspace=ws)
        got = [x.tolist() for x in p] + [so.tolist(), ro.tolist()]
        assert first is None or got == first
        first = got
        assert torch.equal(c.row_state, state) and torch.equal(c.ring, ring)
    _check_tables(c, ref, new, 74)
    assert torch.equal(c.row_state, so) and torch.equal(c.ring, ro)


@gpu
def test_tables_flag_states_that_cannot_be():
    c = _tables_only(4, 20, 4, 16)
    c.row_state[:] = torch.tensor([[-1, 0], [40, 2], [5, 9], [16, 1]], dtype=torch.int32)
    c.block_table[3, 0] = 99                                        # a page that does not exist
    ws = c.alloc_workspace(0)
    p = moba.cache_tables(c, torch.tensor([1, 1, 1, 1], dtype=torch.int32, device="cuda"), 4, workspace=ws)
    assert moba.check_status(ws) == moba.STATUS_BAD_TABLE
    assert p.token_pos.tolist() == [-1, -1, -1, 16]
    c.ring[:] = torch.tensor([5, 2])
    moba.cache_tables(c, torch.tensor([0, 0, 0, 1], dtype=torch.int32, device="cuda"), 1, workspace=ws)
    assert moba.check_status(ws) & moba.STATUS_BAD_TABLE


# ----------------------------------------------------------------------------------------------------- hard conditions
@gpu
def test_refused_rows_are_not_written_and_see_nothing():
    r = Run(3, 6, 8, 2, 1, 64, 16, "e4m3", 3, 2, seed=5)
    plan, want, st = r.tables([40, 0, 10])
    assert st == 0 and r.append(plan, want) == 0
    plan, want, st = r.tables([3, 60, 3])                            # row 1 asks for more pages than are left
    assert st == moba.STATUS_NO_PAGES and want[4] == [1]
    before = r.c.tail_k[1].clone(), r.c.hist[1].clone(), r.c.k.view(torch.uint8).clone()
    assert r.append(plan, want) == 0
    r.check_store()
    assert torch.equal(r.c.tail_k[1].view(torch.int16), before[0].view(torch.int16)) and torch.equal(r.c.hist[1], before[1])
    sel = r.queries(plan, want)                                      # its rows: zeros, -infinity, -1
    dead = [i for i, x in enumerate(want[1]) if x == 1]
    assert (sel[dead] == -1).all()


@gpu
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_nan_and_infinite_tokens_are_stored_as_zero(kind):
    r = Run(2, 20, 8, 2, 2, 64, 16, kind, 0, 3, seed=1)
    plan, want, _ = r.tables([21, 3])
    k, v = r.rand(24, 2, 64), r.rand(24, 2, 64)
    for t, x in ((0, float("nan")), (5, float("inf")), (17, -float("inf")), (22, float("nan"))):
        k[t, 0, 3], v[t, 1, 60] = x, x
    ref_k = torch.where(torch.isfinite(k), k, 0)
    ws = r.c.alloc_workspace(24, 2)
    moba.cache_append(r.c, plan, k.cuda(), v.cuda(), workspace=ws)
    assert moba.check_status(ws) == moba.STATUS_NONFINITE
    r.ref.append(want[0], want[4], ref_k, torch.where(torch.isfinite(v), v, 0), None)
    r.check_store()
    r.queries(plan, want)


@gpu
@pytest.mark.parametrize("W", [0, 4])
def test_a_length_set_back_and_written_again(W):
    """Rejected drafts: lengths go back by up to a block (with the conv by at most 17 - W), across a block's end."""
    B = 32
    r = Run(2, 40, 12, 2, 1, 64, B, "e4m3", W, 3, seed=W)
    r.step([B * 2 + 30, B - 2])
    for back, again in ((5, 4), (12, 13), (13, 1), (1, 30)):
        plan, want, st = r.tables([back, back])
        assert r.append(plan, want) == 0
        r.check_store()
        for i in range(2):                                            # the drafts are rejected: their pages stay
            r.ref.length[i] -= back
        r.c.row_state[:, 0] -= back
        r.step([again, again])


@gpu
@pytest.mark.parametrize("what", ["zero_v", "zero_k", "huge", "tiny", "spread", "denormal"])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("n", [1, 70])        # tiles of 8 and of 128 query rows
def test_scales_of_every_size(what, kind, n):
    r = Run(1, 40, 20, 4, 1, 64, 32, kind, 0, 4, seed=3)
    T = 200
    plan, want, _ = r.tables([T])
    k, v = r.rand(T, 1, 64), r.rand(T, 1, 64)
    blk = (torch.arange(T) // 32)[:, None, None]
    if what == "zero_v":
        v[:] = 0
    elif what == "zero_k":
        k[:] = 0
    elif what == "huge":
        v = (v.float() * 1e30).to(torch.bfloat16)
    elif what == "tiny":
        v, k = (v.float() * 1e-30).to(torch.bfloat16), (k.float() * 1e-30).to(torch.bfloat16)
    elif what == "denormal":                                          # scales at their lower end
        v = (v.float() * 1e-37).to(torch.bfloat16)
    else:                                                             # blocks 2^12 apart from one another
        v = (v.float() * torch.pow(2.0, 12.0 * (blk % 3 - 1))).to(torch.bfloat16)
    assert r.append(plan, want, k, v) == 0
    r.check_store()
    plan, want, _ = r.tables([n])
    assert r.append(plan, want, r.rand(n, 1, 64) * 0 if what in ("zero_v", "tiny", "denormal") else None,
                    r.rand(n, 1, 64) * 0 if what in ("zero_v", "tiny", "denormal") else None) == 0
    q = r.rand(n, 4, 64)
    if what == "denormal":
        # values near 1e-37: what a result loses to the smallest 32-bit numbers is not in the bound; it is small and finite
        ws = r.c.alloc_workspace(n, 4)
        out, lse = moba.cache_attention(r.c, plan, q.cuda(), workspace=ws)
        o, l, mass, size, low = r.ref.attend(want[1], want[2], q)
        assert (out.cpu().double() - o).abs().max() <= 1e-37 and (lse.cpu().double() - l).abs().max() <= 1e-4
        return
    r.queries(plan, want, q)


@gpu
@pytest.mark.parametrize("n", [1, 90])
def test_a_bad_query_spoils_its_own_row_only(n):
    r = Run(1, 40, 20, 4, 1, 64, 32, "e4m3", 0, 4, seed=9)
    plan, want, _ = r.tables([150])
    r.append(plan, want)
    plan, want, _ = r.tables([n])
    r.append(plan, want)
    q = r.rand(n, 4, 64)
    ws = r.c.alloc_workspace(n, 4)
    clean = [x.clone() for x in moba.cache_attention(r.c, plan, q.cuda(), workspace=ws)]
    q[n - 1, 2, 7] = float("nan")
    q[0, 1, 0] = float("inf")
    for sel in (None, moba.cache_route(r.c, plan, q.cuda(), 64, workspace=ws)):
        out, lse = moba.cache_attention(r.c, plan, q.cuda(), sel_idx=sel, workspace=ws)
        bad = torch.zeros((n, 4), dtype=torch.bool)
        bad[n - 1, 2] = bad[0, 1] = True
        assert torch.isnan(out.cpu()[bad]).all() and torch.isnan(lse.cpu()[bad]).all()
        assert torch.isfinite(out.cpu()[~bad].float()).all()
        if sel is None:
            assert torch.equal(out.cpu()[~bad], clean[0].cpu()[~bad]) and torch.equal(lse.cpu()[~bad], clean[1].cpu()[~bad])
    assert moba.check_status(ws) == 0


@gpu
def test_selections_out_of_range_or_out_of_order_are_skipped():
    r = Run(2, 40, 20, 2, 2, 64, 16, "int8", 0, 6, seed=2)
    plan, want, _ = r.tables([100, 90])
    r.append(plan, want)
    plan, want, _ = r.tables([1, 1])
    r.append(plan, want)
    q = r.rand(2, 2, 64)
    own = [100 // 16, 90 // 16]
    sel = torch.tensor([[[0, 2, 2, 1, own[0], -1], [-1, -1, -1, -1, -1, -1]],
                        [[3, own[1], 9, 1000000, -5, -1], [-1, 1, -1, 4, -1, own[1]]]], dtype=torch.int32)
    seen = torch.tensor([[[0, 2, own[0]] + [-1] * 3, [-1] * 6], [[3, own[1]] + [-1] * 4, [1, 4, own[1]] + [-1] * 3]], dtype=torch.int32)
    ws = r.c.alloc_workspace(2, 2)
    out, lse = moba.cache_attention(r.c, plan, q.cuda(), sel_idx=sel.cuda(), workspace=ws)
    assert moba.check_status(ws) == moba.STATUS_BAD_SEL_IDX
    ref = r.ref.attend(want[1], want[2], q, seen)
    cr.check_attention(out.cpu(), lse.cpu(), ref, 64)
    assert (out[0, 1] == 0).all() and lse[0, 1] == -float("inf")


@gpu
@pytest.mark.parametrize("n", [1, 64])
def test_pages_out_of_range_are_skipped(n):
    r = Run(1, 40, 20, 2, 2, 64, 16, "e4m3", 0, 3, seed=4)
    plan, want, _ = r.tables([100])
    r.append(plan, want)
    plan, want, _ = r.tables([n])
    r.append(plan, want)
    q = r.rand(n, 2, 64)
    ws = r.c.alloc_workspace(n, 2)
    good = r.c.block_table.clone()
    r.c.block_table[0, 2], r.c.block_table[0, 4] = -3, 40
    out, lse = moba.cache_attention(r.c, plan, q.cuda(), workspace=ws)
    assert moba.check_status(ws) == moba.STATUS_BAD_TABLE
    every = torch.tensor([[[j if j not in (2, 4) and j <= p // 16 else -1 for j in range(20)]] * 2 for p in want[2]], dtype=torch.int32)
    cr.check_attention(out.cpu(), lse.cpu(), r.ref.attend(want[1], want[2], q, every), 64)
    moba.cache_route(r.c, plan, q.cuda(), 3, workspace=ws)           # ends, whatever it picks
    assert moba.check_status(ws) in (0, moba.STATUS_BAD_TABLE)
    r.c.block_table.copy_(good)
    # a plan that runs ahead of the rows' state
    ahead = moba.CachePlan(plan.cu_new, plan.token_row, plan.token_pos + 1000, plan.slot_map)
    out, lse = moba.cache_attention(r.c, ahead, q.cuda(), workspace=ws)
    assert moba.check_status(ws) == moba.STATUS_BAD_TABLE and (out == 0).all() and torch.isinf(lse).all()
    moba.cache_append(r.c, ahead, r.rand(n, 2, 64).cuda(), r.rand(n, 2, 64).cuda(), workspace=ws)
    assert moba.check_status(ws) == moba.STATUS_BAD_TABLE
    r.check_store()


@gpu
def test_offsets_beyond_32_bits():
    """Pages whose bytes lie past 2^32 in the 8-bit buffers."""
    B, h, d = 128, 8, 128
    n_pages = 34000                                                   # 4.46 GB of keys, as much of values
    r = Run(2, 40, 12, 16, h, d, B, "e4m3", 0, 3, seed=6)
    c = moba.alloc_cache(2, n_pages, 12, h, d, B)
    c.free_pages.copy_(torch.arange(n_pages - 1, -1, -1, dtype=torch.int32))
    r.c, r.check = c, False
    r.ref = cr.RefCache(2, n_pages, 12, h, d, B, "e4m3", 0)
    r.ref.free = cr.deque(range(n_pages - 1, -1, -1))
    for new in ([300, 129], [1, 1], [40, 0]):
        plan, want, st = r.tables(new)
        assert st == 0 and r.append(plan, want) == 0
        ks = c.k_scale
        for i in range(2):                                            # (check_store copies whole buffers: not these)
            for j in range(r.ref.length[i] // B):
                pg = r.ref.pages[i][j]
                code, s = r.ref.block(r.ref.key, i, j)
                assert torch.equal(ks[pg].cpu(), s)
                assert torch.equal(c.k[pg].cpu().float(), code.float())
                r.ref.cents[pg] = c.cent[0, pg].cpu().double() + c.cent[1, pg].cpu().double()
        r.queries(plan, want)


# ---------------------------------------------------------------------------------------------- streams, graphs, the ABI
@gpu
def test_a_generation_step_replays_from_a_graph():
    """One captured step (tables in place, append, route, attention) generates token after token."""
    rows, hq, h, d, B, W, topk = 3, 4, 2, 64, 16, 4, 3
    r = Run(rows, 60, 20, hq, h, d, B, "e4m3", W, topk, seed=8)
    r.step([50, 17, 0])
    new = torch.ones(rows, dtype=torch.int32, device="cuda")
    k, v, q = (torch.zeros((rows, n, d), dtype=torch.bfloat16, device="cuda") for n in (h, h, hq))
    w = r.w.cuda()
    ws = r.c.alloc_workspace(rows, hq)
    state = {n: getattr(r.c, n).clone() for n in ("k", "v", "k_scale", "v_scale", "cent", "tail_k", "tail_v", "hist",
                                                 "block_table", "row_state", "free_pages", "ring")}

    def step():
        plan = moba.cache_tables(r.c, new, rows, workspace=ws)
        moba.cache_append(r.c, plan, k, v, conv_w=w, workspace=ws)
        sel = moba.cache_route(r.c, plan, q, topk, workspace=ws)
        return (plan, sel) + moba.cache_attention(r.c, plan, q, sel_idx=sel, workspace=ws) + \
            moba.cache_attention(r.c, plan, q, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan, sel, out, lse, out_all, lse_all = step()
    for n, x in state.items():                                        # the warm-up step is taken back
        getattr(r.c, n).view(torch.uint8).copy_(x.view(torch.uint8))
    for i in range(20):
        kk, vv, qq = r.rand(rows, h, d), r.rand(rows, h, d), r.rand(rows, hq, d)
        for x, y in ((k, kk), (v, vv), (q, qq)):
            x.copy_(y)
        new.copy_(torch.tensor([1, i % 2, 1]))                         # a row that rests every other step
        graph.replay()
        want = r.ref.tables([1, i % 2, 1], rows)
        for got, exp in zip(plan, want):
            assert got.tolist() == exp
        r.ref.append(want[0], want[4], kk[:], vv, r.w)
        r.check_store()
        n = want[0][-1]
        exp = r.ref.route(want[1], want[2], qq, topk)
        assert torch.equal(sel.cpu()[:n], exp[:n])
        for o, l, e in ((out, lse, exp), (out_all, lse_all, None)):
            ref = r.ref.attend(want[1], want[2], qq, e)
            cr.check_attention(o.cpu()[:n], l.cpu()[:n], [x[:n] for x in ref], d)
    assert moba.check_status(ws) == 0


@gpu
@pytest.mark.parametrize("d,hq,h", [(128, 8, 2), (64, 2, 2)])
def test_a_mixed_step_replays_from_a_graph(d, hq, h):
    """Attention over all blocks of chunks beside single tokens, captured with what comes before and after it: a replay
    gives what a call gives, and the calls around it see its inputs and outputs."""
    r = Run(4, 160, 60, hq, h, d, 64, "e4m3", 0, 3, seed=d)
    plan, want, _ = r.tables([2000, 900, 130, 5])
    assert r.append(plan, want) == 0
    plan, want, _ = r.tables([1, 120, 1, 33], pad=3)
    assert r.append(plan, want) == 0
    T = plan.token_row.shape[0]
    q_in, q, res = (torch.zeros((T, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    ws, ws2 = r.c.alloc_workspace(T, hq), r.c.alloc_workspace(T, hq)

    def step():
        q.copy_(q_in)
        out, lse = moba.cache_attention(r.c, plan, q, workspace=ws)
        res.copy_(out)
        return out, lse

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    real = want[0][-1]
    for _ in range(5):
        q_in.copy_(r.rand(T, hq, d))
        for _ in range(3):
            graph.replay()
        exp, exp_lse = moba.cache_attention(r.c, plan, q_in, workspace=ws2)
        assert moba.check_status(ws) == 0 and moba.check_status(ws2) == 0
        assert torch.equal(out[:real], exp[:real]) and torch.equal(lse[:real], exp_lse[:real])
        assert torch.equal(res[:real], exp[:real])


@gpu
def test_two_streams_with_a_workspace_each():
    """Steps of two caches on two streams at once give what they give alone."""
    a, b = (Run(2, 60, 40, 4, 1, 128, 16, kind, 0, 4, seed=i) for i, kind in enumerate(("e4m3", "int8")))
    jobs = []
    for r in (a, b):
        plan, want, _ = r.tables([300, 100])
        r.append(plan, want)
        plan, want, _ = r.tables([90, 1])
        r.append(plan, want)
        jobs.append((r, plan, want, r.rand(91, 4, 128)))
    alone = []
    for r, plan, want, q in jobs:
        ws = r.c.alloc_workspace(91, 4)
        sel = moba.cache_route(r.c, plan, q.cuda(), 4, workspace=ws)
        alone.append([x.clone() for x in (sel,) + moba.cache_attention(r.c, plan, q.cuda(), sel_idx=sel) + moba.cache_attention(r.c, plan, q.cuda())])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    qs = [q.cuda() for _, _, _, q in jobs]
    torch.cuda.synchronize()
    got = []
    for rep in range(5):
        got = []
        for (r, plan, _, _), q, s in zip(jobs, qs, streams):
            with torch.cuda.stream(s):
                sel = moba.cache_route(r.c, plan, q, 4)
                got.append((sel,) + moba.cache_attention(r.c, plan, q, sel_idx=sel) + moba.cache_attention(r.c, plan, q))
        torch.cuda.synchronize()
        for x, y in zip(got, alone):
            for u, w in zip(x, y):
                assert torch.equal(u, w)


@gpu
def test_binding_refuses_what_does_not_fit():
    c = moba.alloc_cache(2, 10, 4, 2, 64, 16, conv_width=3)
    new = torch.ones(2, dtype=torch.int32, device="cuda")
    plan = moba.cache_tables(c, new, 2)
    ok = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((2, 64, 3), device="cuda")
    with pytest.raises(TypeError):
        moba.cache_append(c, plan, ok.float(), ok, conv_w=w)
    with pytest.raises(ValueError):
        moba.cache_append(c, plan, ok[:1], ok, conv_w=w)
    with pytest.raises(ValueError):
        moba.cache_append(c, plan, torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")[:, ::2], ok, conv_w=w)
    with pytest.raises(ValueError):
        moba.cache_append(c, plan, ok, ok)
    with pytest.raises(ValueError):
        moba.cache_append(c, plan, ok, ok, conv_w=w[..., :2].contiguous())
    with pytest.raises(TypeError):
        moba.cache_tables(c, new.long(), 2)
    with pytest.raises(ValueError):
        moba.cache_tables(c, new[:1], 2)
    with pytest.raises(ValueError):
        moba.cache_tables(c, new, -1)
    with pytest.raises(ValueError):
        moba.cache_tables(c, new, 3, plan=plan)
    with pytest.raises(TypeError):
        moba.cache_route(c, tuple(plan), ok, 2)
    with pytest.raises(ValueError):
        moba.cache_route(c, plan, torch.zeros((2, 2, 128), dtype=torch.bfloat16, device="cuda"), 2)
    for hq, topk in ((3, 2), (2, 0), (2, 65)):
        with pytest.raises((moba.MobaError, RuntimeError)):
            moba.cache_route(c, plan, torch.zeros((2, hq, 64), dtype=torch.bfloat16, device="cuda"), topk)
    with pytest.raises(moba.MobaError):
        moba.cache_route(c, plan, ok, 2, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        moba.cache_attention(c, plan, ok, sel_idx=torch.zeros((1, 2, 2), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        moba.cache_attention(c, plan, ok, lse=torch.zeros((2, 3), device="cuda"))
    other = moba.alloc_cache(3, 10, 4, 2, 64, 16)
    with pytest.raises(ValueError):
        moba.cache_attention(other, plan, ok)
    # nothing to do is no error
    none = moba.cache_tables(c, torch.zeros_like(new), 0)
    empty = ok[:0]
    moba.cache_append(c, none, empty, empty, conv_w=w)
    assert moba.cache_route(c, none, empty, 2).shape == (0, 2, 2)
    assert moba.cache_attention(c, none, empty)[0].shape == (0, 2, 64)


@gpu
@pytest.mark.parametrize("W", [0, 4])
def test_cached_routing_agrees_with_the_prompt_path(W):
    """The same prompt through moba.forward and through the cache: the centroids are the same but for the order of 32-bit
    sums, so selections differ in near ties only."""
    from block_sparse_long_key_b200 import synth
    w = synth.small((700, 333), 4, 2, 64, 32, 6, conv_width=W, seed=4)
    x = {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in synth.make_inputs(w, with_dout=False).items()}
    out, lse, sel, _ = moba.forward(x["q"], x["k"], x["v"], x["cu_seqlens"], 32, 6, conv_w=x.get("conv_w"))
    c = moba.alloc_cache(2, 40, 30, 2, 64, 32, conv_width=W)
    plan = moba.cache_tables(c, torch.tensor([700, 333], dtype=torch.int32, device="cuda"), 1033)
    moba.cache_append(c, plan, x["k"], x["v"], conv_w=x.get("conv_w"))
    got = moba.cache_route(c, plan, x["q"], 6)
    same = (got == sel).all(-1)
    assert same.float().mean() > 0.999
    o, l = moba.cache_attention(c, plan, x["q"], sel_idx=got)
    # e4m3 keeps keys to 2^-4: scores move by about 2^-4 / sqrt(3) / sqrt(64) |q| |k| ~ 0.04 rms, outputs likewise
    d = (o.float() - out.float())[same]
    assert d.pow(2).mean().sqrt() < 0.1 * out.float().pow(2).mean().sqrt()
    assert (l - lse)[same].abs().max() < 0.5


@gpu
@pytest.mark.parametrize("cu", [[0, 90], [5, 90], [-7, 90], [90, 3], [200, 400]])
def test_plans_that_contradict_themselves_stay_in_bounds(cu):
    """First tokens that cannot be: calls end, nothing behind the buffers is touched (what they compute is not defined)."""
    r = Run(1, 40, 20, 8, 2, 64, 16, "e4m3", 0, 3, seed=4)
    plan, want, _ = r.tables([100])
    r.append(plan, want)
    plan, want, _ = r.tables([90])
    assert r.append(plan, want) == 0
    q = r.rand(90, 8, 64).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    odd = moba.CachePlan(torch.tensor(cu, **i32), plan.token_row, plan.token_pos, plan.slot_map)
    k, v = (torch.zeros((90, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = r.c.alloc_workspace(90, 8)
    guard = torch.full((92, 8, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    sel = moba.cache_route(r.c, odd, q, 3, workspace=ws)
    moba.cache_attention(r.c, odd, q, workspace=ws, out=guard[1:91])
    moba.cache_attention(r.c, odd, q, sel_idx=sel, workspace=ws, out=guard[1:91])
    moba.check_status(ws)
    assert (guard[0] == 3).all() and (guard[91] == 3).all()
    tail = r.c.tail_k.clone()
    moba.cache_append(r.c, odd, k, v, workspace=ws)
    moba.check_status(ws)
    if cu == [0, 90]:
        return
    few = moba.CachePlan(torch.tensor([cu[0], cu[1]], **i32), plan.token_row[:3].contiguous(), plan.token_pos[:3].contiguous(),
                         plan.slot_map[:3].contiguous())
    moba.cache_append(r.c, few, k[:3].contiguous(), v[:3].contiguous(), workspace=ws)
    moba.cache_attention(r.c, few, q[:3].contiguous(), workspace=ws)
    moba.check_status(ws)
