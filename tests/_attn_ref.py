"""The softmax-layer operators in 64 bits, written from their definitions, each with the error that its kernel is
allowed: every rounding to bf16 counts half a step (2^-8 of the value), what stays in 32 bits a few of its steps."""
from __future__ import annotations

import math

import torch

H = 2.0 ** -8      # half a step of bf16, relative
S = 2.0 ** -14     # a few hundred steps of fp32: sums of d products, exponentials, row sums
TINY = 2.0 ** -126  # relative steps hold for normal numbers of bf16 and fp32: below the smallest, a weight may be 0
F64 = torch.float64


def doc_list(B, T, cu):
    if cu is None:
        return [(b * T, T) for b in range(B)]
    cu = [int(x) for x in cu]
    return [(a, b - a) for a, b in zip(cu[:-1], cu[1:])]


def attn(q, k, v, scale, cu=None, dO=None):
    """dict of (value, tolerance): o, lse [Hq, B*T], and with dO also dq, dk, dv."""
    B, T, Hq, d = q.shape
    Hk = k.shape[2]
    G, dev = Hq // Hk, q.device
    flat = lambda x: x.reshape(B * T, -1, d).to(F64)
    q, k, v = flat(q), flat(k), flat(v)
    zeros = lambda x: (torch.zeros_like(x), torch.zeros_like(x))
    out = {"o": zeros(q), "lse": zeros(torch.empty((Hq, B * T), dtype=F64, device=dev))}
    if dO is not None:
        dO = flat(dO)
        out.update(dq=zeros(q), dk=zeros(k), dv=zeros(k))
    for at, n in doc_list(B, T, cu):
        if n == 0:
            continue
        r = slice(at, at + n)
        mask = torch.ones((n, n), dtype=torch.bool, device=dev).tril()
        for h in range(Hq):
            kk, vv, qq = k[r, h // G], v[r, h // G], q[r, h]
            x = (qq @ kk.T * scale).masked_fill(~mask, -math.inf)
            amp = (qq.abs() @ kk.abs().T * scale).masked_fill(~mask, 0)
            lse = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[:, None])
            o = p @ vv
            out["o"][0][r, h] = o
            out["o"][1][r, h] = H * o.abs() + (H + S) * (p @ vv.abs()) + TINY * vv.abs().sum(0)
            out["lse"][0][h, r] = lse
            out["lse"][1][h, r] = 2.0 ** -17 * (1 + lse.abs() + amp.amax(1))
            if dO is None:
                continue
            g = dO[r, h]
            dp = g @ vv.T
            delta = (g * o).sum(1, keepdim=True)
            # delta is taken from the o that the forward rounded
            d_err = H * (g * o).abs().sum(1, keepdim=True)
            ds = p * (dp - delta)
            ds_err = H * ds.abs() + p * (d_err + S * (g.abs() @ vv.abs().T + delta.abs())) + TINY * (dp - delta).abs()
            out["dq"][0][r, h] = scale * (ds @ kk)
            out["dq"][1][r, h] = scale * (ds_err @ kk.abs())
            out["dk"][0][r, h // G] += scale * (ds.T @ qq)
            out["dk"][1][r, h // G] += scale * (ds_err.T @ qq.abs())
            out["dv"][0][r, h // G] += p.T @ g
            out["dv"][1][r, h // G] += (H + S) * (p.T @ g.abs()) + TINY * g.abs().sum(0)
    for x in ("dq", "dk", "dv"):
        if x in out:
            out[x][1].add_(H * out[x][0].abs())
    return {x: (a.view(B, T, -1, d) if x != "lse" else a, b.view(B, T, -1, d) if x != "lse" else b)
            for x, (a, b) in out.items()}


def positions(B, T, cu, device):
    if cu is None:
        return torch.arange(T, dtype=F64, device=device).expand(B, T)
    pos = torch.zeros(T, dtype=F64, device=device)
    for at, n in doc_list(B, T, cu):
        pos[at:at + n] = torch.arange(n, dtype=F64, device=device)
    return pos[None]


def rotation(pos, rotary, base, d, interleaved):
    """The d x d rotation of each token, [B, T, d, d]: y_rotated = R y."""
    R = torch.eye(d, dtype=F64, device=pos.device).repeat(*pos.shape, 1, 1)
    for i in range(rotary // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
        ang = pos * base ** (-2.0 * i / rotary)
        R[..., a, a] = R[..., b, b] = ang.cos()
        R[..., a, b] = -ang.sin()
        R[..., b, a] = ang.sin()
    return R


def norm(x, w, R, eps, dy=None):
    """(y, tolerance), or with dy ((dx, tolerance), (dw, tolerance)); R as from rotation()."""
    x, w = x.to(F64), w.to(F64)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r
    fine = 2.0 ** -18
    if dy is None:
        y = torch.einsum("btij,bthj->bthi", R, n * w)
        return y, H * y.abs() + fine * (n * w).abs().amax(-1, keepdim=True)
    back = torch.einsum("btji,bthj->bthi", R, dy.to(F64))
    h = back * w
    m = (h * n).mean(-1, keepdim=True)
    dx = r * (h - n * m)
    size = r * (h.abs().amax(-1, keepdim=True) + n.abs().amax(-1, keepdim=True) * (h * n).abs().mean(-1, keepdim=True))
    dw, dw_size = (back * n).sum((0, 1, 2)), (back.abs().amax(-1, keepdim=True) * n.abs()).sum((0, 1, 2))
    return (dx, H * dx.abs() + 4 * fine * size), (dw, 2.0 ** -16 * dw_size)


def cached(q, kc, vc, pages, lens, tree, scale):
    """(o, tolerance), (lse, tolerance) [B, T, Hq]; positions without a valid page are not seen."""
    B, T, Hq, d = q.shape
    n_pages, page, Hk, _ = kc.shape
    G, dev = Hq // Hk, q.device
    o = torch.zeros((B, T, Hq, d), dtype=F64, device=dev)
    ot, l, lt = torch.zeros_like(o), torch.full((B, T, Hq), -math.inf, dtype=F64, device=dev), None
    lt = torch.zeros_like(l)
    for b in range(B):
        n = int(lens[b])
        end = min(n + T, pages.shape[1] * page) if n >= 0 else 0
        t = torch.arange(end, device=dev)
        pg = pages[b].long()[t // page] if end else t
        good = (pg >= 0) & (pg < n_pages)
        row = pg.clamp(0, n_pages - 1) * page + t % page
        see = torch.zeros((T, end), dtype=torch.bool)
        for i in range(T):
            for j in range(end):
                if j < n:
                    see[i, j:n] = True
                    break
            for j in range(max(n, 0), end):
                e = j - n
                see[i, j] = e <= i if tree is None else bool((int(tree[b, i]) >> e) & 1)
        see = see.to(dev) & good[None]
        if not end:
            continue
        kk = kc.view(-1, Hk, d)[row].to(F64).masked_fill(~see.any(0)[:, None, None], 0)
        vv = vc.view(-1, Hk, d)[row].to(F64).masked_fill(~see.any(0)[:, None, None], 0)
        some = see.any(1)
        for h in range(Hq):
            qq = q[b, :, h].to(F64)
            x = (qq @ kk[:, h // G].T * scale).masked_fill(~see, -math.inf)
            lse = torch.logsumexp(x, 1)
            p = torch.where(some[:, None], torch.exp(x - torch.where(some, lse, 0)[:, None]), 0)
            amp = (qq.abs() @ kk[:, h // G].abs().T * scale).amax(1)
            o[b, :, h] = p @ vv[:, h // G]
            ot[b, :, h] = H * o[b, :, h].abs() + (H + S) * (p @ vv[:, h // G].abs())
            l[b, :, h] = lse
            lt[b, :, h] = 2.0 ** -17 * (1 + torch.where(some, lse.abs(), 0) + amp)
    return (o, ot), (l, lt)


def check(name, got, want):
    ref, tol = want
    got = got.to(F64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    same = got == ref   # infinities
    bad = ~(((got - ref).abs() <= tol + TINY) | same)
    assert not bool(bad.any()), \
        f"{name}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}: " \
        f"{float(got[bad][0])} for {float(ref[bad][0])} +- {float(tol[bad][0])}"
