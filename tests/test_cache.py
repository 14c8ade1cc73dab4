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
        self.hq, self.topk, self.scale = h_q, topk, scale
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
            self.check_store()
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
