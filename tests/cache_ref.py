"""A plain 64-bit paged cache: lists of tokens per row, one row at a time.

Shares no code with the package.  Keys and values are what the cache keeps of
them: bf16 tokens, and for complete blocks the 8-bit values times their scale.
"""
import math
from collections import deque

import torch

QMAX = {"e4m3": 448.0, "int8": 127.0}
F8 = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def bf16(x):
    return x.float().to(torch.bfloat16)


class RefCache:
    def __init__(self, rows, n_pages, max_blocks, h_kv, d, B, kind, conv_width):
        self.rows, self.n_pages, self.max_blocks, self.h, self.d, self.B = rows, n_pages, max_blocks, h_kv, d, B
        self.kind, self.W = kind, conv_width
        self.cents = {}   # page -> centroids as the cache under test holds them, where routing is to follow those
        self.free = deque(range(n_pages))
        self.pages = [[] for _ in range(rows)]
        self.length = [0] * rows
        self.raw = [torch.zeros((0, h_kv, d), dtype=torch.bfloat16) for _ in range(rows)]
        self.key = [torch.zeros((0, h_kv, d), dtype=torch.bfloat16) for _ in range(rows)]
        self.val = [torch.zeros((0, h_kv, d), dtype=torch.bfloat16) for _ in range(rows)]

    def tables(self, new_len, T):
        """(cu, token_row, token_pos, slot, refused rows); advances the state."""
        B = self.B
        cu, row, pos, slot, refused = [0], [], [], [], []
        avail, asked = len(self.free), 0
        give_back = []
        for r, n in enumerate(new_len):
            if n < 0:
                give_back += self.pages[r]
                self.pages[r], self.length[r] = [], 0
                for x in (self.raw, self.key, self.val):
                    x[r] = x[r][:0]
                cu.append(cu[-1])
                continue
            blocks = -(-(self.length[r] + n) // B)
            need = max(0, blocks - len(self.pages[r]))
            ok = blocks <= self.max_blocks
            if ok:
                asked += need
                ok = need == 0 or asked <= avail
            fits = cu[-1] + n <= T
            first = cu[-1]
            cu.append(min(T, first + n))
            if not fits and n > 0:
                ok = False
            if ok:
                self.pages[r] += [self.free.popleft() for _ in range(need)]
            else:
                refused.append(r)
            for i in range(cu[-1] - first):
                p = self.length[r] + i
                row.append(r)
                pos.append(p if ok else -1)
                slot.append(self.pages[r][p // B] * B + p % B if ok else -1)
            if ok:
                self.length[r] += n
        self.free.extend(give_back)
        pad = T - len(row)
        return cu, row + [-1] * pad, pos + [-1] * pad, slot + [-1] * pad, refused

    def append(self, cu, refused, k, v, w):
        for r in range(self.rows):
            a, b = cu[r], cu[r + 1]
            if a == b or r in refused:
                continue
            old = self.length[r] - (b - a)
            for x, new in ((self.raw, k[a:b]), (self.val, v[a:b])):
                x[r] = torch.cat([x[r][:old], new])
            self.val[r] = torch.where(torch.isfinite(self.val[r]), self.val[r], 0)
            key = self.raw[r][old:].double()
            if self.W:
                z = torch.zeros_like(key)
                line = torch.cat([torch.zeros((self.W, self.h, self.d), dtype=torch.float64), self.raw[r].double()])
                for l in range(self.W):
                    z += w[:, :, l].double() * line[self.W + old - l:self.W + old - l + (b - a)]
                key = key + z / (1 + torch.exp(-z))
            key = bf16(key)
            key = torch.where(torch.isfinite(key), key, 0)
            self.key[r] = torch.cat([self.key[r][:old], key])

    def block(self, x, r, j):
        """(codes, scale) of complete block j of a row's keys or values: [h, B, d], [h]."""
        t = x[r][j * self.B:(j + 1) * self.B].float().transpose(0, 1)
        s = (t.abs().amax((1, 2)) * (torch.tensor(1.0) / QMAX[self.kind])).clamp_min(2.0 ** -126)
        y = t / s[:, None, None]
        if self.kind == "e4m3":
            return y.clamp(-448, 448).to(torch.float8_e4m3fn), s
        return torch.round(y).clamp(-127, 127).to(torch.int8), s

    def centroid(self, r, j):
        c = (self.key[r][j * self.B:(j + 1) * self.B].double().sum(0) / self.B).float()
        hi = c.to(torch.bfloat16)
        return hi, (c - hi.float()).to(torch.bfloat16)

    def held(self, r):
        """The row's keys and values as the cache holds them, float64 [len, h, d]."""
        out = []
        for x in (self.key, self.val):
            parts = []
            for j in range(self.length[r] // self.B):
                c, s = self.block(x, r, j)
                parts.append((c.float().double() * s.double()[:, None, None]).transpose(0, 1))
            parts.append(x[r][self.length[r] // self.B * self.B:].double())
            out.append(torch.cat(parts))
        return out

    def route(self, row, pos, q, topk):
        T, hq, _ = q.shape
        g = hq // self.h
        sel = torch.full((T, hq, topk), -1, dtype=torch.int32)
        cents = {}
        for t in range(T):
            if row[t] < 0 or pos[t] < 0:
                continue
            r, own = row[t], pos[t] // self.B
            if r not in cents:
                cs = [self.cents.get(self.pages[r][j]) for j in range(self.length[r] // self.B)]
                cents[r] = torch.stack(cs) if cs else None
            for h in range(hq):
                got = []
                if own:
                    x = (cents[r][:own, h // g] * q[t, h].double()).sum(-1)
                    x = torch.where(torch.isnan(x), -math.inf, x)
                    got = sorted(torch.sort(x, descending=True, stable=True).indices[:topk - 1].tolist())
                got.append(own)
                sel[t, h, :len(got)] = torch.tensor(got, dtype=torch.int32)
        return sel

    def attend(self, row, pos, q, sel=None):
        """out, lse, and the bounds' parts: sum p|v|, the score error scale, keys x largest |v|; all float64."""
        T, hq, d = q.shape
        g = hq // self.h
        out = torch.zeros((T, hq, d), dtype=torch.float64)
        lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
        mass = torch.zeros((T, hq, d), dtype=torch.float64)
        size = torch.zeros((T, hq), dtype=torch.float64)
        low = torch.zeros((T, hq), dtype=torch.float64)
        held = {}
        for t in range(T):
            if row[t] < 0 or pos[t] < 0:
                continue
            r = row[t]
            if r not in held:
                held[r] = self.held(r)
            for h in range(hq):
                if sel is None:
                    at = list(range(pos[t] + 1))
                else:
                    at = [p for j in sel[t, h].tolist() if j >= 0 for p in range(j * self.B, min((j + 1) * self.B, pos[t] + 1))]
                if not at:
                    continue
                k, v = held[r][0][at, h // g], held[r][1][at, h // g]
                s = (k * q[t, h].double()).sum(-1) / math.sqrt(d)
                p = torch.softmax(s, 0)
                out[t, h] = (p[:, None] * v).sum(0)
                mass[t, h] = (p[:, None] * v.abs()).sum(0)
                lse[t, h] = torch.logsumexp(s, 0)
                size[t, h] = (k.abs() * q[t, h].double().abs()).sum(-1).max() / math.sqrt(d)
                low[t, h] = len(at) * v.abs().max()
        return out, lse, mass, size, low


def check_attention(out, lse, ref, d, what=""):
    """Output against the reference.  The output is rounded to bf16 once (half a step, 2^-8 of the value).  A weight
    p = exp(s - m) is off by its rounding to fp16 (2^-11), the scores by the rounding of d products and sums and of
    the few steps to the exponent in 32 bits: delta = (d + 16) 2^-24 sum|q k| / sqrt(d); p by about delta + 2^-20
    (the exponential).  Both the weights and their sum carry that, hence twice.

    fp16 also has a smallest step, 2^-24, so a weight is off by up to 2^-25 however small it is.  Weights carry the
    block's V scale and the largest one is at least 2^7, so with w_i = p_i vs_i c, c >= 2^7 / max(p vs), that moves the
    output by at most sum_i 2^-25 |v8_i| / c <= 2^-32 sum_i |v8_i| max(p vs) <= 2^-32 n max|v|: |v8_i| is at most the
    largest code, and that times the largest scale is max|v|."""
    o, l, mass, size, low = ref
    delta = (d + 16) * 2.0 ** -24 * size + 2.0 ** -20
    err = (out.double() - o).abs()
    tol = 2.0 ** -8 * o.abs() + (1 + 2.0 ** -7) * mass * (2.0 ** -11 + 2 * torch.expm1(2 * delta))[..., None] + 2.0 ** -32 * low[..., None] + 1e-38
    assert torch.isfinite(out.double()).all(), what
    assert (err <= tol).all(), (what, float((err / tol).max()))
    empty = torch.isinf(l)
    assert torch.equal(torch.isinf(lse.double()), empty), what
    gap = (lse.double() - l).abs()[~empty]
    assert (gap <= (2 * delta + 2.0 ** -23 * l.abs())[~empty] + 1e-6).all(), (what, float(gap.max()))
