"""The 64-bit references of the softmax layer against automatic differentiation and against differences, and the
entry points' refusals, none of which needs a GPU."""
import ctypes

import pytest
import torch

import _attn_ref as ref
from chunked_linear_attention_bounded_gb300 import bdla
from chunked_linear_attention_bounded_gb300.build import build

F64 = torch.float64


def _rand(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed + sum(shape)), dtype=F64)


def test_attention_gradient_reference_against_autograd_and_differences():
    cu = [0, 3, 3, 10]
    q, k, v, dO = _rand(1, 10, 4, 8), _rand(1, 10, 2, 8, seed=1), _rand(1, 10, 2, 8, seed=2), _rand(1, 10, 4, 8, seed=3)
    got = ref.attn(q, k, v, 0.3, cu, dO)

    def loss(q, k, v):
        total = 0
        for at, n in ref.doc_list(1, 10, cu):
            kk, vv = (x[0, at:at + n].repeat_interleave(2, 1) for x in (k, v))
            x = torch.einsum("ihd,jhd->hij", q[0, at:at + n], kk) * 0.3
            x = x.masked_fill(~torch.ones(n, n, dtype=torch.bool).tril(), -torch.inf)
            total = total + (torch.einsum("hij,jhd->ihd", x.softmax(-1), vv) * dO[0, at:at + n]).sum()
        return total

    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    loss(*leaves).backward()
    for x, n in zip(leaves, ("dq", "dk", "dv")):
        torch.testing.assert_close(got[n][0], x.grad, rtol=1e-10, atol=1e-10)
    u = _rand(1, 10, 2, 8, seed=9)
    e = 1e-5
    diff = ((ref.attn(q, k + e * u, v, 0.3, cu)["o"][0] - ref.attn(q, k - e * u, v, 0.3, cu)["o"][0]) * dO).sum() / (2 * e)
    torch.testing.assert_close((got["dk"][0] * u).sum(), diff, rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("inter", [False, True])
def test_norm_gradient_reference_against_autograd(inter):
    x, w, dy = _rand(2, 3, 2, 64), _rand(64, seed=5), _rand(2, 3, 2, 64, seed=6)
    R = ref.rotation(ref.positions(2, 3, None, "cpu") + 11, 32, 100.0, 64, inter)
    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    y = torch.einsum("btij,bthj->bthi", R, a / torch.sqrt((a * a).mean(-1, keepdim=True) + 1e-3) * b)
    torch.testing.assert_close(y.detach(), ref.norm(x, w, R, 1e-3)[0])
    (y * dy).sum().backward()
    (dx, _), (dw, _) = ref.norm(x, w, R, 1e-3, dy)
    torch.testing.assert_close(dx, a.grad)
    torch.testing.assert_close(dw, b.grad)
    torch.testing.assert_close(R @ R.transpose(-1, -2), torch.eye(64, dtype=F64).expand_as(R))


def test_cached_reference_is_the_last_rows_of_whole_attention():
    """A chain of drafts over a shuffled cache is causal attention over the sequence."""
    n, T, page = 13, 4, 3
    q, k, v = _rand(1, n + T, 4, 8), _rand(1, n + T, 2, 8, seed=1), _rand(1, n + T, 2, 8, seed=2)
    order = torch.randperm(9, generator=torch.Generator().manual_seed(4))[:6]
    kc, vc = torch.full((9, page, 2, 8), float("nan"), dtype=F64), torch.full((9, page, 2, 8), float("nan"), dtype=F64)
    for t in range(n + T):
        kc[order[t // page], t % page] = k[0, t]
        vc[order[t // page], t % page] = v[0, t]
    (o, _), (l, _) = ref.cached(q[:, n:], kc, vc, order[None].int(), [n], None, 0.4)
    want = ref.attn(q, k, v, 0.4)
    torch.testing.assert_close(o, want["o"][0][:, n:])
    torch.testing.assert_close(l[0].T, want["lse"][0][:, n:])


# ------------------------------------------------------------------ refusals
FAKE = 1 << 20   # non-NULL, aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    build()
    return bdla.lib()


def _norm(L, d=(1, 4, 4, 2, 64), out=FAKE, ws=FAKE, ws_bytes=1 << 30, gdt=0, bwd=False, **kw):
    a = dict(q=FAKE, k=FAKE, q_token=256, q_head=64, k_token=128, k_head=64, wq=FAKE, wk=FAKE, positions=None,
             cu_seqlens=None, base=1e4, eps=1e-6, rotary=64, interleaved=0, n_docs=0)
    a.update(kw)
    args = bdla.QkNormArgs(*[a[n] for n, _ in bdla.QkNormArgs._fields_])
    if bwd:
        return L.bdla_qk_norm_bwd(args, FAKE, FAKE, gdt, out, FAKE, FAKE, FAKE, bdla.AttnDims(*d), ws, ws_bytes, None)
    return L.bdla_qk_norm(args, out, FAKE, bdla.AttnDims(*d), None)


@pytest.mark.parametrize("bwd", [False, True])
def test_norm_refusals(L, bwd):
    E = bdla
    no = lambda **kw: _norm(L, bwd=bwd, **kw)
    assert no(q=None) == no(wk=None) == no(out=None) == E.ERR_NULL
    assert no(d=(1, 4, 4, 2, 96)) == E.ERR_UNSUPPORTED
    assert no(d=(1, 4, 5, 2, 64)) == no(d=(0, 4, 4, 2, 64)) == no(d=(1, -1, 4, 2, 64)) == E.ERR_SHAPE
    assert no(d=(2, 1 << 30, 4, 2, 64)) == E.ERR_TOO_LARGE
    assert no(rotary=8) == no(rotary=80) == no(rotary=-16) == E.ERR_SHAPE
    assert no(q_token=252) == no(k_head=4) == no(q=FAKE + 8) == no(out=FAKE + 4) == E.ERR_ALIGN
    assert no(eps=-1.0) == no(eps=float("nan")) == no(base=0.5) == no(base=float("inf")) == E.ERR_RANGE
    assert no(cu_seqlens=FAKE, n_docs=0) == no(cu_seqlens=FAKE, n_docs=2, d=(2, 4, 4, 2, 64)) == E.ERR_SHAPE
    if bwd:
        assert no(gdt=5) == E.ERR_DTYPE
        assert no(ws=None) == no(ws_bytes=100) == no(ws=FAKE + 8) == E.ERR_WORKSPACE


def test_attn_refusals(L):
    E = bdla
    D = E.AttnDims

    def fwd(d=D(1, 4, 4, 2, 64), q=FAKE, cu=None, n=0, scale=0.125, ws=FAKE, wsb=1 << 30, o=FAKE):
        return L.bdla_attn_fwd(q, FAKE, FAKE, cu, n, scale, o, FAKE, d, ws, wsb, None)

    def bwd(d=D(1, 4, 4, 2, 64), q=FAKE, cu=None, n=0, scale=0.125, ws=FAKE, wsb=1 << 30, o=FAKE):
        return L.bdla_attn_bwd(q, FAKE, FAKE, o, FAKE, FAKE, cu, n, scale, FAKE, FAKE, FAKE, d, ws, wsb, None)

    for f in (fwd, bwd):
        assert f(q=None) == f(o=None) == E.ERR_NULL
        assert f(q=FAKE + 2) == E.ERR_ALIGN
        assert f(scale=0.0) == f(scale=-1.0) == f(scale=float("inf")) == f(scale=float("nan")) == E.ERR_RANGE
        assert f(d=D(1, 4, 4, 3, 64)) == f(d=D(1, 4, 0, 0, 64)) == f(cu=FAKE, n=0) == E.ERR_SHAPE
        assert f(d=D(2, 4, 4, 2, 64), cu=FAKE, n=2) == E.ERR_SHAPE
        assert f(d=D(1, 4, 4, 2, 256)) == f(d=D(65536, 1, 4, 2, 64)) == E.ERR_UNSUPPORTED
        assert f(d=D(4, 1 << 29, 4, 2, 64)) == E.ERR_TOO_LARGE
        assert f(ws=None) == f(wsb=255) == E.ERR_WORKSPACE
        assert f(d=D(1, 1 << 30, 512, 1, 64)) == E.ERR_TOO_LARGE      # (128 tokens, head) units are a grid extent
    assert L.bdla_workspace_bytes_attn(E.ATTN_BWD, D(1, 100, 4, 2, 64), 0, 0) >= 256 + 1600
    assert L.bdla_workspace_bytes_attn(E.ATTN_BWD, D(1, 100, 4, 3, 64), 0, 0) == 0
    assert L.bdla_workspace_bytes_attn(99, D(1, 100, 4, 2, 64), 0, 0) == 0


def test_cache_refusals(L):
    E = bdla
    D = E.AttnDims

    def cache(k=FAKE, v=FAKE, pages=FAKE, lens=FAKE, n_pages=4, page=16, max_pages=2):
        return E.CacheArgs(k, v, pages, lens, n_pages, page, max_pages)

    def append(c=cache(), d=D(2, 3, 2, 2, 64), k=FAKE, ws=FAKE, wsb=1 << 30):
        return L.bdla_cache_append(k, FAKE, c, None, None, d, ws, wsb, None)

    def attend(c=cache(), d=D(2, 3, 4, 2, 64), k=FAKE, ws=FAKE, wsb=1 << 30, scale=0.1, tree=None, o=FAKE):
        return L.bdla_attn_cached(k, c, tree, scale, o, FAKE, d, ws, wsb, None)

    for f in (append, attend):
        assert f(k=None) == f(c=cache(lens=None)) == f(c=cache(pages=None)) == f(c=cache(v=None)) == E.ERR_NULL
        assert f(k=FAKE + 8) == f(c=cache(k=FAKE + 8)) == E.ERR_ALIGN
        assert f(c=cache(page=0)) == f(c=cache(n_pages=-1)) == f(c=cache(max_pages=-1)) == E.ERR_SHAPE
        assert f(c=cache(page=65537)) == E.ERR_UNSUPPORTED
        assert f(c=cache(page=65536, max_pages=40000)) == E.ERR_TOO_LARGE
        assert f(ws=None) == f(wsb=10) == E.ERR_WORKSPACE
    assert attend(d=D(2, 65, 4, 2, 64)) == E.ERR_UNSUPPORTED
    assert attend(d=D(2, 0, 4, 2, 64)) == E.ERR_SHAPE
    assert attend(scale=0.0) == E.ERR_RANGE
    assert attend(tree=FAKE + 4) == E.ERR_ALIGN
    assert attend(o=None) == E.ERR_NULL


def test_python_refusals():
    """CPU tensors and wrong ranks are refused before the library is reached."""
    q = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16)
    w = torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        bdla.attn_fwd(q, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        bdla.qk_norm(q, q, w, w)
    with pytest.raises(ValueError, match="CUDA"):
        bdla.attn_cached(q, q, q, torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        bdla.cache_append([0], q, q, q, None, None)
