"""Long documents and long caches, by the norm of the error.

A bound of each entry by the worst case grows with the length, to several percent of an entry's size at 2000 keys.  The
roundings of single weights are independent: the square of their sum's error is the sum of their squares.  A rounding to
bf16 is off by at most H of the value, evenly in both directions, so its mean square is at most H^2 / 3 of the value's;
over the 10^5 and more entries of a tensor the mean is what is met.  What stays in fp32 (exponentials, sums over a row or
a column) counts S of the norms of the sum and of its terms.  The bounds come to 0.3 to 0.4% of the norm, so that a key in
a hundred left out or taken twice (10% in a simulation) does not pass."""
import pytest
import torch

import _attn_ref as ref
from chunked_linear_attention_bounded_gb300 import bdla

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
H, S = ref.H, ref.S
THIRD = H * H / 3


def _rn(g, *s):
    return torch.randn(s, generator=g, device="cuda").to(BF16)


def _bound(want, squares):
    """Of the error's norm, `squares` being the summed squares of what was rounded on its way into the sums."""
    size = float((want * want).sum())
    return (THIRD * (size + squares)) ** 0.5 + S * (size ** 0.5 + squares ** 0.5)


def _bounded(name, got, want, squares):
    err, bound = float((got.to(F64) - want).norm()), _bound(want, squares)
    assert err <= bound, f"{name}: error {err:.4g}, bound {bound:.4g}, norm {float(want.norm()):.4g}"
    assert bound <= 5e-3 * float(want.norm()), f"{name}: the bound says nothing ({bound:.4g} of {float(want.norm()):.4g})"


LONG = [
    # lens, Hq, Hk, d, spread: one document of 16K with a CTA a key head, ragged ones with a CTA a query head
    ((16384,), 4, 2, 128, 2),
    ((9001, 5, 4987), 3, 1, 64, 2),
    ((12345,), 2, 1, 128, 1),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(str(x) for x in c))
def test_long_documents(case):
    lens, Hq, Hk, d, spread = case
    T, G, scale = sum(lens), Hq // Hk, d ** -0.5
    g = torch.Generator("cuda").manual_seed(T)
    q, k, v, dO = _rn(g, 1, T, Hq, d) * spread, _rn(g, 1, T, Hk, d), _rn(g, 1, T, Hk, d), _rn(g, 1, T, Hq, d)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    zeros = lambda h: torch.zeros((T, h, d), dtype=F64, device="cuda")
    want = dict(o=zeros(Hq), dq=zeros(Hq), dk=zeros(Hk), dv=zeros(Hk))
    lse = torch.zeros((Hq, T), dtype=F64, device="cuda")
    sq = dict.fromkeys(want, 0.0)
    at = 0
    for n in lens:
        for h in range(Hq):
            kk, vv = k[0, at:at + n, h // G].to(F64), v[0, at:at + n, h // G].to(F64)
            for r0 in range(0, n, 2048):
                r1 = min(n, r0 + 2048)
                r, c = slice(at + r0, at + r1), slice(at, at + r1)
                qq, gg, kb, vb = q[0, r, h].to(F64), dO[0, r, h].to(F64), kk[:r1], vv[:r1]
                x = (qq @ kb.T * scale).masked_fill(~torch.ones((r1 - r0, r1), dtype=torch.bool, device="cuda").tril(r0), -torch.inf)
                lse[h, r] = torch.logsumexp(x, 1)
                p = torch.exp(x - lse[h, r, None])
                o = p @ vb
                dp, delta = gg @ vb.T, (gg * o).sum(1, keepdim=True)
                ds = p * (dp - delta) * scale
                want["o"][r, h], want["dq"][r, h] = o, ds @ kb
                want["dk"][c, h // G] += ds.T @ qq
                want["dv"][c, h // G] += p.T @ gg
                # weights to bf16; ds to bf16; delta from the rounded o (mean square of its error a row: e2)
                p2, ds2, e2 = p * p, ds * ds, (gg * o).square().sum(1, keepdim=True) * scale ** 2
                sq["o"] += float((p2 @ vb.square()).sum())
                sq["dv"] += float((p2.T @ gg.square()).sum())
                sq["dq"] += float((ds2 @ kb.square()).sum() + (e2 * (p @ kb).square()).sum())
                sq["dk"] += float((ds2.T @ qq.square()).sum() + ((p2 * e2).T @ qq.square()).sum())
        at += n
    ws = bdla.Workspace(256, "cuda")
    o, l = bdla.attn_fwd(q, k, v, cu_seqlens=cu, ws=ws)
    got = dict(o=o, **dict(zip(("dq", "dk", "dv"), bdla.attn_bwd(q, k, v, want["o"][None].to(BF16), lse.float(), dO,
                                                                 cu_seqlens=cu, ws=ws))))
    assert ws.read_device_status() == bdla.OK
    assert float((l.to(F64) - lse).abs().max()) <= 2.0 ** -17 * (1 + float(lse.abs().max()) + 3 * spread * d ** 0.5)
    for n, w in want.items():
        _bounded(n, got[n][0], w, sq[n])


@pytest.mark.parametrize("T,Hq,tree", [(1, 16, False), (4, 8, False), (61, 8, True)])
def test_long_caches(T, Hq, tree):
    """Few rows a key head (pieces joined) and many (the tensor-memory kernel), contexts far longer than a piece, and a
    table that is wider than either needs."""
    lens, page, Hk, d = (60001, 20000, 3), 48, 2, 128
    B, G, scale = len(lens), Hq // Hk, 128 ** -0.5
    g = torch.Generator("cuda").manual_seed(T)
    need = [-(-(n + T) // page) for n in lens]
    order = torch.randperm(sum(need), generator=g, device="cuda").int()
    table = torch.full((B, 2 * max(need)), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(need):
        table[b, :n] = order[sum(need[:b]):sum(need[:b + 1])]
    kc, vc = _rn(g, sum(need), page, Hk, d), _rn(g, sum(need), page, Hk, d)
    q = _rn(g, B, T, Hq, d) * 2
    bits = None
    if tree:   # each sees itself and the even ones before it
        bits = torch.tensor([[(1 << i) | (0x5555555555555555 & ((1 << i) - 1)) for i in range(T)]] * B, device="cuda")
    ws = bdla.Workspace(256, "cuda")
    o, lse = bdla.attn_cached(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), tree=bits, ws=ws)
    assert ws.read_device_status() == bdla.OK
    for b, n in enumerate(lens):
        kk, vv = (x[table[b, :need[b]].long()].flatten(0, 1)[:n + T].to(F64) for x in (kc, vc))
        see = torch.ones((T, n + T), dtype=torch.bool, device="cuda").tril(n)
        if tree:
            j = torch.arange(T, device="cuda")
            see[:, n:] = (j[None] <= j[:, None]) & ((j[None] % 2 == 0) | (j[None] == j[:, None]))
        want, squares = torch.zeros((T, Hq, d), dtype=F64, device="cuda"), 0.0
        for h in range(Hq):
            x = (q[b, :, h].to(F64) @ kk[:, h // G].T * scale).masked_fill(~see, -torch.inf)
            l = torch.logsumexp(x, 1)
            p = torch.exp(x - l[:, None])
            want[:, h] = p @ vv[:, h // G]
            squares += float((p.square() @ vv[:, h // G].square()).sum())
            assert float((lse[b, :, h].to(F64) - l).abs().max()) <= 2.0 ** -17 * (1 + float(l.abs().max()) + 6 * d ** 0.5)
        if T * Hq * d >= 10000:
            _bounded(f"sequence {b}", o[b], want, squares)
        else:   # the mean square of few entries may be met by half again
            assert float((o[b].to(F64) - want).norm()) <= 1.5 * _bound(want, squares)
