"""The paged 8-bit cache at the ends of what its calls allow, against the plain 64-bit cache (cache_ref.py): lengths that
go back, values of extreme size, steps without tokens."""
import ctypes

import pytest
import torch

import cache_ref as cr
from block_sparse_long_key_b200 import moba
from test_cache import FAKE, L, Run, _plan, _route_alone, _route_exact, _struct  # noqa: F401  (L: the built library)

gpu = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------- lengths that go back
@pytest.mark.parametrize("W,back", [(0, -1), (4, -1), (4, 14), (8, 10), (2, 16), (0, 17)])
def test_lengths_cannot_go_back_further_than_the_history(L, W, back):  # noqa: F811
    ref, pr = ctypes.byref(_struct(conv_width=W, hist=FAKE, set_back=back)), ctypes.byref(_plan())
    assert L.moba_cache_workspace_size(ref, 4, 2) == 0
    assert L.moba_cache_append(ref, pr, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == moba.MOBA_EINVAL
    fits = _struct(conv_width=W, hist=FAKE, set_back=17 - max(W, 1))
    assert L.moba_cache_workspace_size(ctypes.byref(fits), 4, 2) > 0


def _take_back(r, back):
    """Sets the rows' lengths back by `back` tokens each (their pages stay)."""
    for i, s in enumerate(back):
        r.ref.length[i] -= s
    r.c.row_state[:, 0] -= torch.tensor(back, dtype=torch.int32, device="cuda")


def _write(r, new):
    plan, want, st = r.tables(new)
    assert st == 0 and r.append(plan, want) == 0


@gpu
@pytest.mark.parametrize("d,B", [(64, 16), (128, 16), (128, 128)])
@pytest.mark.parametrize("W", [2, 4, 8])
def test_part_of_a_step_is_taken_back(W, d, B):
    """Drafts of n tokens of which n - s are accepted, for every s the header allows: the keys that follow are those of a
    cache that never saw the rejected ones.  Fewer and more drafts than the conv is wide; blocks end inside."""
    jobs = [(n, s) for n in (2, 3, 4, 5, 9, 16, 17, 40) for s in range(1, min(n - 1, 17 - W, B) + 1)]
    rows = len(jobs)
    r = Run(rows, rows * (140 // B + 4), 140 // B + 4, 2, 2, d, B, "e4m3", W, 3, seed=W + d)
    _write(r, [(5 * i) % (B + 3) + (i % 3 > 0) * 7 for i in range(rows)])
    _write(r, [n for n, _ in jobs])
    _take_back(r, [s for _, s in jobs])
    _write(r, [1] * rows)                                  # (Run.append compares what is held, bit for bit)
    _write(r, [i % 4 for i in range(rows)])
    _write(r, [B if i % 2 else 3 for i in range(rows)])


@gpu
@pytest.mark.parametrize("W", [0, 3])
def test_lengths_go_back_more_than_once(W):
    """Each time to no less than the longest length so far less what the header allows."""
    B = 16
    r = Run(3, 60, 16, 2, 1, 64, B, "int8", W, 3, seed=11)
    _write(r, [37, 16, 5])
    longest = list(r.ref.length)
    for new, back in (((6, 9, 1), (4, 2, 1)), ((1, 1, 1), (3, 5, 2)), ((2, 3, 20), (4, 3, 9)), ((5, 1, 1), (5, 4, 6)),
                      ((1, 40, 2), (0, 13, 5))):
        _write(r, new)
        longest = [max(a, b) for a, b in zip(longest, r.ref.length)]
        back = [min(s, n - max(m - min(B, 17 - W), 0)) for s, n, m in zip(back, r.ref.length, longest)]
        _take_back(r, back)
        _write(r, [1, 2, 1])
        longest = [max(a, b) for a, b in zip(longest, r.ref.length)]


@gpu
@pytest.mark.parametrize("W,back", [(4, 0), (4, 3), (8, 9), (2, 15)])
def test_the_history_holds_what_going_back_needs(W, back):
    """Of a step's raw keys the last W - 1 + set_back, each at its position mod 16; the others stay as they were."""
    h, d, B, n = 2, 128, 16, (1, 2, 5, 30, 16)
    c = moba.alloc_cache(len(n), 40, 4, h, d, B, conv_width=W, set_back=back)
    c.hist.fill_(-9)
    k = torch.randn((sum(n), h, d), generator=torch.Generator().manual_seed(W)).to(torch.bfloat16)
    plan = moba.cache_tables(c, torch.tensor(n, dtype=torch.int32, device="cuda"), sum(n))
    moba.cache_append(c, plan, k.cuda(), k.cuda(), conv_w=torch.zeros((h, d, W), device="cuda"))
    want, first = torch.full_like(c.hist, -9).cpu(), 0
    for r, x in enumerate(n):
        for p in range(max(0, x - (W - 1 + back)), x):
            want[r, p % 16] = k[first + p]
        first += x
    assert torch.equal(c.hist.cpu(), want)


# ---------------------------------------------------------------------------------------------------------- magnitudes
@gpu
@pytest.mark.parametrize("what", ["tiny_cent", "tiny_query", "small_cent", "small_query", "both", "tiny_beside_zero",
                                  "subnormal_cent", "subnormal_query"])
def test_routing_of_small_magnitudes(what):
    """Scores far inside the range of 32 bits whose squares are not: the blocks are still those of the exact scores."""
    g = torch.Generator().manual_seed(5)
    nb, h, d, B, T, hq, topk = 1500, 2, 64, 16, 120, 8, 17
    cent = torch.randn((nb, h, d), generator=g).double()
    q = torch.randn((T, hq, d), generator=g).to(torch.bfloat16)
    if what in ("tiny_cent", "tiny_beside_zero"):
        cent = cent * 1e-24
    elif what == "tiny_query":
        q = (q.float() * 1e-24).to(torch.bfloat16)
    elif what == "small_cent":                                 # squares just below, and just inside, the normal range
        cent = cent * 2.0 ** -65
    elif what == "small_query":
        q = (q.float() * 2.0 ** -65).to(torch.bfloat16)
    elif what == "both":
        cent, q = cent * 2.0 ** -70, (q.float() * 2.0 ** 70).to(torch.bfloat16)
    elif what == "subnormal_cent":
        cent, q = cent * 1e-39, (q.float() * 1e20).to(torch.bfloat16)
    elif what == "subnormal_query":
        cent, q = cent * 1e20, (q.float() * 1e-39).to(torch.bfloat16)
    if what == "tiny_beside_zero":
        cent[::3] = 0
    own = nb - 1
    sel, held = _route_alone(cent, q, own * B + 5, B, topk)
    assert torch.equal(sel, _route_exact(held, q, own, topk))


@gpu
@pytest.mark.parametrize("d,B", [(64, 16), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_centroids_of_the_largest_keys(kind, d, B):
    """Means that 32 bits hold, of tokens whose sums they do not; and signs that cancel."""
    r = Run(1, 8, 6, 2, 2, d, B, kind, 0, 2, seed=d + B)
    T = 3 * B + 3
    plan, want, _ = r.tables([T])
    k = r.rand(T, 2, d)
    top = torch.finfo(torch.bfloat16).max
    k[:B] = top
    k[B:2 * B] = (1e38 * (1 + 0.1 * k[B:2 * B].float().clamp(-1, 1))).to(torch.bfloat16)
    k[2 * B:3 * B:2], k[2 * B + 1:3 * B:2] = top, -top
    assert r.append(plan, want, k, r.rand(T, 2, d)) == 0      # (Run.append compares the centroids with the 64-bit means)
    cent = r.c.cent.float()
    assert torch.isfinite(cent).all(dim=(2, 3))[:, r.ref.pages[0][:3]].all()
    assert (cent[0, r.ref.pages[0][0]] == top).all() and (cent[:, r.ref.pages[0][2]] == 0).all()


@gpu
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,n", [(4, 1), (96, 1), (96, 3)])   # tiles of 8 and of 128 query rows
@pytest.mark.parametrize("power", [-27, -90, -106, -112, -118])
def test_values_far_below_one(kind, hq, n, power):
    """V of every binary size from 1 down to the end of the normal range, one block of 16 keys of it and nothing else to
    sum.  The block's scale is about 3 2^power / QMAX; scales below 2^-100 take a factor of their own (`rest`)."""
    B, d = 16, 64
    r = Run(1, 8, 6, hq, 1, d, B, kind, 0, 2, seed=hq - power)
    plan, want, _ = r.tables([B])
    k, v = r.rand(B, 1, d), r.rand(B, 1, d)
    v = (v.float() * 2.0 ** power).to(torch.bfloat16)
    assert r.append(plan, want, k, v) == 0
    plan, want, _ = r.tables([n])
    none = torch.zeros((n, 1, d), dtype=torch.bfloat16)
    assert r.append(plan, want, none, none) == 0
    q = r.rand(n, hq, d)
    ws = r.c.alloc_workspace(n, hq)
    out, lse = moba.cache_attention(r.c, plan, q.cuda(), workspace=ws)
    assert moba.check_status(ws) == 0
    ref = list(r.ref.attend(want[1], want[2], q))
    # check_attention's bound for weights below fp16's normal range, 2^-32 sum |v8_i| max(p vs), with vs as the kernels
    # take it for the reference, at least 2^-100: then n QMAX 2^-100 stands in place of n max|v|, where that is more.
    # Weights may be rounded to fp16 twice, before and after that factor: 2^-11 of the mass each.  lse is a sum of two
    # numbers of up to 2^7, rounded to 2^-18 each.
    ref[4] = torch.maximum(ref[4], torch.full_like(ref[4], (B + n) * cr.QMAX[kind] * 2.0 ** -100))
    o, l, mass, size, low = ref
    out, lse = out.cpu(), lse.cpu()
    delta = (d + 16) * 2.0 ** -24 * size + 2.0 ** -20
    tol = 2.0 ** -8 * o.abs() + 2.0 ** -133 + (1 + 2.0 ** -7) * mass * (2.0 ** -10 + 2 * torch.expm1(2 * delta))[..., None] + \
        2.0 ** -32 * low[..., None]
    err = (out.double() - o).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert ((lse.double() - l).abs() <= 2 * delta + 2.0 ** -17).all()
    # And it is an answer, not zeros: at 2^-118 the heaviest of 16 weights is about 2^7 2^-25 (the factor is 2^-25.2 for
    # e4m3), each is off by 2^-24 / sqrt(12) rms, so the outputs by 2^-25.8 sqrt(16) / 2^-18.2 = 0.02 of their rms.
    assert err.pow(2).mean().sqrt() <= 0.05 * o.pow(2).mean().sqrt()


@gpu
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,n", [(4, 1), (96, 1), (4, 30)])   # tiles of 8, of 128 and of 16 query rows
@pytest.mark.parametrize("where", ["first", "last", "every_other", "tail"])
def test_blocks_of_zeros_beside_large_values(kind, hq, n, where):
    """A value of zero counts in the softmax's sum like any other, whatever the size of the others: V of 1e13, of 1 and of
    1e-20, with whole blocks of zeros before, behind and between."""
    B, d, held = 32, 64, 6 * 32 + 11
    for size in (1e13, 1.0, 1e-20):
        r = Run(1, 20, 14, hq, 1, d, B, kind, 0, 8, seed=hq + n)
        plan, want, _ = r.tables([held])
        v = (r.rand(held, 1, d).float() * size).to(torch.bfloat16)
        blk = torch.arange(held) // B
        v[{"first": blk < 2, "last": (blk == 4) | (blk == 5), "every_other": blk % 2 == 0, "tail": blk == 6}[where]] = 0
        assert r.append(plan, want, None, v) == 0
        plan, want, _ = r.tables([n])
        new = torch.zeros((n, 1, d)) if where == "tail" else r.rand(n, 1, d).float() * size
        assert r.append(plan, want, None, new.to(torch.bfloat16)) == 0
        r.queries(plan, want)


@gpu
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,n", [(4, 1), (96, 1)])
@pytest.mark.parametrize("held", [64, 75, 90])                 # whole blocks, and a partial one of 11 or 26 tokens
def test_values_near_the_largest(kind, hq, n, held):
    """V of 1e38, in blocks and in the partial one, and one new token of 1e10 (scales 2^93 apart; the limit is 2^100)."""
    r = Run(1, 12, 10, hq, 1, 64, 32, kind, 0, 3, seed=held)
    plan, want, _ = r.tables([held])
    v = (r.rand(held, 1, 64).float().clamp(-3.3, 3.3) * 1e38).to(torch.bfloat16)
    assert r.append(plan, want, None, v) == 0
    plan, want, _ = r.tables([n])
    assert r.append(plan, want, None, (r.rand(n, 1, 64).float() * 1e10).to(torch.bfloat16)) == 0
    r.queries(plan, want)


@gpu
@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("power", [0, -60, -118, -124, -130])
def test_converted_keys_of_small_magnitudes(W, power):
    """Keys, and the conv's products, down to the end of the range: still the rounding of the 64-bit value.  With blocks of
    128 the tail holds all tokens of these rows."""
    rows, n, h, d, B = 12, 250, 4, 128, 128
    g = torch.Generator().manual_seed(W - power)
    k = (torch.randn((rows * n, h, d), generator=g) * 2.0 ** power).to(torch.bfloat16)
    w = torch.rand((h, d, W), generator=g) - 0.5
    c = moba.alloc_cache(rows, 2 * rows, 2, h, d, B, conv_width=W)
    plan = moba.cache_tables(c, torch.full((rows,), n, dtype=torch.int32, device="cuda"), rows * n)
    moba.cache_append(c, plan, k.cuda(), torch.zeros_like(k).cuda(), conv_w=w.cuda())
    got = c.tail_k.cpu().permute(0, 1, 3, 2, 4).reshape(rows, 2 * B, h, d)[:, :n]
    x = torch.cat([torch.zeros((rows, W, h, d), dtype=torch.float64), k.double().reshape(rows, n, h, d)], 1)
    z = sum(w[:, :, l].double() * x[:, W - l:W - l + n] for l in range(W))
    want = (x[:, W:] + z / (1 + torch.exp(-z))).float().to(torch.bfloat16)
    assert torch.equal(got.float(), want.float()), int((got.float() != want.float()).sum())


@gpu
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("d,B,hq,n", [(128, 16, 8, 19), (64, 32, 3, 60), (128, 128, 40, 3), (64, 16, 96, 1), (64, 32, 3, 9)])
def test_small_weights_beside_a_sharp_softmax(kind, d, B, hq, n):
    """Keys with a millionth of the weight, where the heaviest key's value is near zero in a channel: in whole blocks and
    in the partial one, for tiles of every size."""
    for seed in range(4):
        r = Run(2, 400 // B + 30, 400 // B + 10, hq, 1, d, B, kind, 0, 4, seed=seed, scale=4.0)
        for held in (B // 2 + 1, 3 * B):
            plan, want, _ = r.tables([held, 2 * B])
            assert r.append(plan, want) == 0
            plan, want, _ = r.tables([n, n + 1])
            k, v = r.rand(2 * n + 1, 1, d), r.rand(2 * n + 1, 1, d)
            assert r.append(plan, want, k, v) == 0
            r.queries(plan, want)


@gpu
@pytest.mark.parametrize("hq,n", [(4, 1), (96, 1), (4, 30)])
def test_lse_does_not_depend_on_the_values(hq, n):
    """V scales on either side of where the kernels take another path, and of their ends, set in the cache by hand."""
    B, d, held = 16, 64, 5 * 16 + 3
    r = Run(1, 12, 9, hq, 1, d, B, "int8", 0, 4, seed=n)
    plan, want, _ = r.tables([held])
    assert r.append(plan, want) == 0
    plan, want, _ = r.tables([n])
    assert r.append(plan, want) == 0
    q = r.rand(n, hq, d)
    o, lse_ref, mass, size, low = r.ref.attend(want[1], want[2], q)
    delta = (d + 16) * 2.0 ** -24 * size + 2.0 ** -20
    for edge in (2.0 ** -126, 2.0 ** -100, 2.0 ** -40, 1.0, 2.0 ** 40):
        x = torch.tensor(edge)
        for scale in (torch.nextafter(x, torch.tensor(0.0)), x, torch.nextafter(x, torch.tensor(1e30))):
            for pages in (r.ref.pages[0], r.ref.pages[0][1:3]):            # all blocks, and two among ordinary ones
                r.c.v_scale.fill_(1.0)
                r.c.v_scale[pages] = scale.item()
                ws = r.c.alloc_workspace(n, hq)
                out, lse = moba.cache_attention(r.c, plan, q.cuda(), workspace=ws)
                assert moba.check_status(ws) == 0
                # M and log2 l are rounded to 2^-18 each where they are as large as 2^7
                assert ((lse.cpu().double() - lse_ref).abs() <= 2 * delta + 2.0 ** -17).all(), (edge, scale.item(), len(pages))


# ------------------------------------------------------------------------------------------- beside the prompt path
@gpu
@pytest.mark.parametrize("W", [1, 4])
def test_cached_keys_beside_those_of_the_prompt_path(W):
    """moba_forward forms k' in 32 bits, the cache rounds the 64-bit value: they differ by one step of bf16 at most (and
    what 32-bit sums lose), and seldom.  With blocks of 128 the last two blocks' keys can be read back from the tail."""
    B, n, h, d = 128, 200, 2, 64
    g = torch.Generator().manual_seed(W)
    k, v = (torch.randn((n, h, d), generator=g).to(torch.bfloat16) for _ in range(2))
    w = torch.rand((h, d, W), generator=g) - 0.5
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    prompt = moba.forward(k.cuda(), k.cuda(), v.cuda(), cu, B, 2, conv_w=w.cuda())[3].cpu().double()
    c = moba.alloc_cache(1, 4, 4, h, d, B, conv_width=W)
    plan = moba.cache_tables(c, torch.tensor([n], dtype=torch.int32, device="cuda"), n)
    moba.cache_append(c, plan, k.cuda(), v.cuda(), conv_w=w.cuda())
    cached = c.tail_k[0].cpu().double().permute(0, 2, 1, 3).reshape(2 * B, h, d)[:n]
    x = torch.cat([torch.zeros((W, h, d), dtype=torch.float64), k.double()])
    taps = [x[W - l:W - l + n] for l in range(W)]
    z = sum(w[:, :, l].double() * taps[l] for l in range(W))
    size = sum(w[:, :, l].double().abs() * taps[l].abs() for l in range(W))
    exact = k.double() + z / (1 + torch.exp(-z))
    assert torch.equal(cached, exact.float().to(torch.bfloat16).double())
    # 32 bits: W + 2 roundings of the sum, 2 + |z| of the exponential and a few of the quotient, relative 2^-24 each
    off = (1.2 * W + 18) * 2.0 ** -24 * size + 2.0 ** -23 * k.double().abs()
    assert ((prompt - cached).abs() <= 2.0 ** -7 * exact.abs() + off).all()
    assert (prompt == cached).double().mean() > 0.99


# --------------------------------------------------------------------------------------------------- steps of nothing
@gpu
def test_steps_of_padding_only_between_others():
    """Every token is padding: nothing is written, and the calls behind keep their status."""
    r = Run(2, 20, 8, 4, 2, 64, 16, "e4m3", 2, 3, seed=7)
    r.step([40, 9])
    for T in (1, 5, 300):
        plan, want, _ = r.tables([0, 0], pad=T)
        assert want[1] == [-1] * T
        assert r.append(plan, want) == 0
        r.queries(plan, want)
        plan, want, st = r.tables([200, 0])                        # more than there are blocks for
        assert st == moba.STATUS_NO_PAGES
    r.step([1, 1])


@gpu
def test_a_step_without_tokens_leaves_a_clean_status():
    c = moba.alloc_cache(2, 10, 4, 2, 64, 16)
    none = moba.cache_tables(c, torch.zeros(2, dtype=torch.int32, device="cuda"), 0)
    empty = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    for call in (lambda ws: moba.cache_append(c, none, empty, empty, workspace=ws),
                 lambda ws: moba.cache_route(c, none, empty, 2, workspace=ws),
                 lambda ws: moba.cache_attention(c, none, empty, workspace=ws)):
        ws = c.alloc_workspace(0, 2)
        ws.fill_(255)
        call(ws)
        assert moba.check_status(ws) == 0


def test_a_step_without_tokens_checks_the_workspace_it_is_given(L):  # noqa: F811
    ref, none = ctypes.byref(_struct()), ctypes.byref(_plan(total_new=0, token_row=None, token_pos=None, slot_map=None))
    for ws, size, rc in ((FAKE + 128, 1 << 20, moba.MOBA_EALIGN), (FAKE, 128, moba.MOBA_EWORKSPACE), (None, 0, moba.MOBA_OK)):
        assert L.moba_cache_append(ref, none, None, None, None, ws, size, None) == rc
        assert L.moba_cache_route(ref, none, None, 2, 4, None, ws, size, None) == rc
        assert L.moba_cache_attention(ref, none, None, 2, None, 1, None, None, ws, size, None) == rc


def test_more_tokens_than_a_step_may_have_are_refused(L):  # noqa: F811
    ref, big = ctypes.byref(_struct()), _plan(total_new=1 << 24)     # T h_kv d = 2^31
    assert L.moba_cache_tables(ref, FAKE, None, None, ctypes.byref(big), FAKE, 1 << 40, None) == moba.MOBA_EINVAL


# ------------------------------------------------------------------------------------- calls that no other test makes
@gpu
@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_nan_and_infinite_keys_under_the_conv(kind, W):
    """They reach the keys of the W - 1 tokens behind as well, in the same step and from the history in the next."""
    r = Run(2, 30, 8, 2, 2, 64, 16, kind, W, 3, seed=W)
    for new, bad in (([21, 3], ((0, float("nan")), (15, float("inf")), (20, -float("inf")))), ([1, 14], ((1, float("nan")),)),
                     ([2, 1], ())):
        plan, want, _ = r.tables(new)
        T = sum(new)
        k = r.rand(T, 2, 64)
        for t, x in bad:
            k[t, 0, 3], k[t, 1, 60] = x, -x
        reached = bad or W > 2          # the last bad key is at position 20 of row 0, whose third step begins at 22
        assert r.append(plan, want, k) == (moba.STATUS_NONFINITE if reached else 0)
    r.queries(plan, want)


@gpu
def test_a_plan_is_written_again_and_a_planned_state_is_used():
    """One set of plan tensors for every step, roomier than the steps; the state after a step planned into other tensors
    and the step then done with those."""
    r = Run(3, 40, 12, 4, 2, 64, 16, "e4m3", 3, 3, seed=13)
    c, T = r.c, 40
    i32 = dict(dtype=torch.int32, device="cuda")
    plan = moba.CachePlan(torch.empty(4, **i32), *(torch.empty(T, **i32) for _ in range(3)))
    state, ring = torch.empty_like(c.row_state), torch.empty_like(c.ring)
    then = moba.Cache(rows=3, n_pages=40, max_blocks=12, h_kv=2, head_dim=64, block_size=16, conv_width=3, k=c.k, v=c.v,
                      k_scale=c.k_scale, v_scale=c.v_scale, cent=c.cent, tail_k=c.tail_k, tail_v=c.tail_v, hist=c.hist,
                      block_table=c.block_table, row_state=state, free_pages=c.free_pages, ring=ring, set_back=14)
    for new in ([33, 1, 0], [1, 20, 17], [3, -1, 1], [1, 5, 1]):
        want = r.ref.tables(new, T)
        ws = c.alloc_workspace(T, 4)
        assert moba.cache_tables(c, torch.tensor(new, **i32), T, row_state_out=state, ring_out=ring, plan=plan, workspace=ws) is plan
        assert moba.check_status(ws) == 0
        for got, exp in zip(plan, want):
            assert got.tolist() == exp
        k, v, q = r.rand(T, 2, 64), r.rand(T, 2, 64), r.rand(T, 4, 64)
        moba.cache_append(then, plan, k.cuda(), v.cuda(), conv_w=r.w.cuda(), workspace=ws)
        assert moba.check_status(ws) == 0
        r.ref.append(want[0], want[4], k, v, r.w)
        r.c = then
        r.check_store()
        r.queries(plan, want, q)
        r.c = c
        c.row_state.copy_(state), c.ring.copy_(ring)


@gpu
@pytest.mark.parametrize("W,chunk", [(4, 65536), (0, 30000)])
def test_a_long_prompt(W, chunk):
    """64K tokens of 16 heads, whole and in chunks: routing against the centroids that are held, attention of some queries
    against the tokens that are held, both in 64 bits."""
    n, h, d, B, topk = 65536, 16, 64, 32, 32
    g = torch.Generator(device="cuda").manual_seed(W)
    rand = lambda: torch.randn((n, h, d), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    k, v, q = rand(), rand(), rand()
    w = torch.rand((h, d, W), generator=g, device="cuda") - 0.5 if W else None
    c = moba.alloc_cache(1, n // B + 3, n // B + 3, h, d, B, conv_width=W)
    for first in range(0, n, chunk):
        m = min(chunk, n - first)
        at = slice(first, first + m)
        plan = moba.cache_tables(c, torch.tensor([m], dtype=torch.int32, device="cuda"), m)
        ws = c.alloc_workspace(m, h)
        moba.cache_append(c, plan, k[at], v[at], conv_w=w, workspace=ws)
        sel = moba.cache_route(c, plan, q[at], topk, workspace=ws)
        got = [moba.cache_attention(c, plan, q[at], sel_idx=s, workspace=ws) for s in (sel, None)]
        assert moba.check_status(ws) == 0
        done = (first + m) // B
        pages = c.block_table[0, :done].long()
        cent = c.cent[0, pages].double() + c.cent[1, pages].double()
        x8 = [(a.view(torch.uint8)[pages].view(a.dtype).double() * s[pages].double()[:, :, None, None]).transpose(1, 2).reshape(-1, h, d)
              for a, s in ((c.k, c.k_scale), (c.v, c.v_scale))]
        left = (first + m) % B
        keys, vals = (torch.cat([x, t[0, done % 2, :, :left].double().transpose(0, 1)]) for x, t in zip(x8, (c.tail_k, c.tail_v)))
        for t in sorted({0, 1, m // 3, m // 2 + 17, m - B - 1, m - 1}):
            p = first + t
            own = p // B
            s = torch.einsum("jhd,hd->hj", cent[:own], q[p].double())
            top = torch.sort(s, dim=-1, descending=True, stable=True).indices[:, :topk - 1].sort(-1).values
            want = torch.cat([top, torch.full((h, 1), own, device="cuda")], 1)
            want = torch.nn.functional.pad(want, (0, topk - want.shape[1]), value=-1)
            assert torch.equal(sel[t].long(), want), (first, t)
            score = torch.einsum("lhd,hd->hl", keys[:p + 1], q[p].double()) / d ** 0.5
            size = torch.einsum("lhd,hd->hl", keys[:p + 1].abs(), q[p].double().abs()).amax(-1, keepdim=True) / d ** 0.5
            block = torch.arange(p + 1, device="cuda") // B
            for (out, lse), rows in zip(got, (want, None)):
                z = score
                if rows is not None:
                    z = torch.where((rows[:, None] == block[None, :, None]).any(-1), score, -torch.inf)
                pr = torch.softmax(z, -1)
                o, mass = (torch.einsum("hl,lhd->hd", pr, y) for y in (vals[:p + 1], vals[:p + 1].abs()))
                low = (p + 1) * vals[:p + 1].abs().amax((0, 2))[:, None]
                ref = [x[None].cpu() for x in (o, torch.logsumexp(z, -1), mass, size[:, 0], low[:, 0])]
                cr.check_attention(out[t:t + 1].cpu(), lse[t:t + 1].cpu(), ref, d, (first, t, rows is None))
