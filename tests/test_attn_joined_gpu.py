"""attn_bwd is the gradient at the o and lse that it is handed: p = e^{s - lse} and delta = dO . o also where those were
joined with what the call does not see (a sink in the denominator, attention over another set of keys)."""
import math

import pytest
import torch

import _attn_ref as ref
from chunked_linear_attention_bounded_gb300 import bdla

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
H, S = ref.H, ref.S


def _gradient(q, k, v, o, lse, dO, scale, lens):
    """(value, tolerance) of dq, dk, dv, in 64 bits from the o and lse given.

    The kernel may put the weights over their sum for the weights where that sum is within H of 1 (H |ds|), and its own
    sum of p dp for delta within the rounding of o (H sum |dO o|); it rounds ds (H) and p (H) once, and its outputs."""
    Hq, G = q.shape[2], q.shape[2] // k.shape[2]
    q, k, v, o, dO = (x[0].to(F64) for x in (q, k, v, o, dO))
    lse = lse.to(F64)
    out = {n: (torch.zeros_like(x), torch.zeros_like(x)) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    at = 0
    for n in lens:
        r = slice(at, at + n)
        at += n
        mask = torch.ones((n, n), dtype=torch.bool, device=q.device).tril()
        for h in range(Hq):
            kk, vv, qq, g = k[r, h // G], v[r, h // G], q[r, h], dO[r, h]
            p = torch.exp(qq @ kk.T * scale - lse[h, r, None]).masked_fill(~mask, 0)
            dp, delta = g @ vv.T, (g * o[r, h]).sum(1, keepdim=True)
            ds = p * (dp - delta)
            err = 2 * H * ds.abs() + p * (H * (g * o[r, h]).abs().sum(1, keepdim=True) +
                                          S * (g.abs() @ vv.abs().T + delta.abs())) + ref.TINY * (dp - delta).abs()
            out["dq"][0][r, h] = scale * (ds @ kk)
            out["dq"][1][r, h] = scale * (err @ kk.abs())
            out["dk"][0][r, h // G] += scale * (ds.T @ qq)
            out["dk"][1][r, h // G] += scale * (err.T @ qq.abs())
            out["dv"][0][r, h // G] += p.T @ g
            out["dv"][1][r, h // G] += (H + S) * (p.T @ g.abs()) + ref.TINY * g.abs().sum(0)
    for a, b in out.values():
        b.add_(H * a.abs())
    return {n: (a[None], b[None]) for n, (a, b) in out.items()}


def _inputs(d, lens, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF16)
    T = sum(lens)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    return rn(1, T, 4, d), rn(1, T, 2, d), rn(1, T, 2, d), rn(1, T, 4, d), cu, g


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("other", ["nothing", "faint sink", "sink", "strong sink", "keys", "keys of large values"])
def test_gradient_at_a_joined_output(d, other):
    lens = (1, 100, 300, 129)
    q, k, v, dO, cu, g = _inputs(d, lens, len(other))
    scale = d ** -0.5
    want = ref.attn(q, k, v, scale, cu.cpu())
    o, lse = want["o"][0], want["lse"][0]
    size = {"nothing": -math.inf, "faint sink": -9.0, "sink": 1.0, "strong sink": 8.0, "keys": 2.0, "keys of large values": -6.0}[other]
    lse2 = size + torch.randn(lse.shape, generator=g, device="cuda", dtype=F64)
    amount = {"keys": 1.0, "keys of large values": 1000.0}.get(other, 0.0)
    o2 = amount * torch.randn(o.shape, generator=g, device="cuda", dtype=F64)
    both = torch.logaddexp(lse, lse2)
    share = lambda x: torch.exp(x - both).T[None, :, :, None]
    o, lse = (o * share(lse) + o2 * share(lse2)).to(BF16), both.float()
    ws = bdla.Workspace(256, "cuda")
    got = bdla.attn_bwd(q, k, v, o, lse, dO, cu_seqlens=cu, ws=ws)
    assert ws.read_device_status() == bdla.OK
    for (n, w), x in zip(_gradient(q, k, v, o, lse, dO, scale, lens).items(), got):
        ref.check(n, x, w)
