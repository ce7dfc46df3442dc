"""Arguments that bdla_qk_norm_append refuses on the host, before any launch (fake pointers are never read)."""
import pytest

from chunked_linear_attention_bounded_gb300 import bdla
from chunked_linear_attention_bounded_gb300.build import build

P = 1 << 20


@pytest.fixture(scope="module")
def L():
    build()
    return bdla.lib()


def _call(L, dims=(3, 5, 8, 2, 128), q=P, k=P, v=P, wq=P, wk=P, positions=None, cu=None, rows=P, counts=P, qn=P, ws=P,
          ws_bytes=1 << 20, strides=(1536, 128, 1536, 128), v_strides=(1536, 128), base=1e4, eps=1e-6, rotary=128, n_docs=0,
          kc=P, vc=P, pages=P, lens=P, n_pages=9, page=16, max_pages=4):
    a = bdla.QkNormArgs(q, k, *strides, wq, wk, positions, cu, base, eps, rotary, 0, n_docs)
    return L.bdla_qk_norm_append(a, v, *v_strides, bdla.CacheArgs(kc, vc, pages, lens, n_pages, page, max_pages), rows, counts,
                                 qn, bdla.AttnDims(*dims), ws, ws_bytes, None)


def test_refusals(L):
    for dims, want in (((0, 5, 8, 2, 128), bdla.ERR_SHAPE), ((3, -1, 8, 2, 128), bdla.ERR_SHAPE),
                       ((3, 5, 8, 3, 128), bdla.ERR_SHAPE), ((3, 5, 8, 0, 128), bdla.ERR_SHAPE),
                       ((3, 5, 8, 2, 96), bdla.ERR_UNSUPPORTED), ((65536, 1, 8, 2, 128), bdla.ERR_UNSUPPORTED),
                       ((60000, 60000, 8, 2, 128), bdla.ERR_TOO_LARGE)):
        assert _call(L, dims=dims) == want, dims
    for x in ("k", "v", "wq", "wk", "qn", "kc", "vc", "pages", "lens"):
        assert _call(L, **{x: None}) == bdla.ERR_NULL, x
    for x in ("q", "k", "v", "wq", "wk", "qn", "kc", "vc"):
        assert _call(L, **{x: P + 8}) == bdla.ERR_ALIGN, x
    for i in range(4):
        assert _call(L, strides=tuple(1536 + (4 if x == i else 0) for x in range(4))) == bdla.ERR_ALIGN
    assert _call(L, v_strides=(1540, 128)) == _call(L, v_strides=(1536, 132)) == bdla.ERR_ALIGN
    for bad in (dict(rotary=24), dict(rotary=144), dict(rotary=-16), dict(n_pages=-1), dict(page=0), dict(max_pages=-1)):
        assert _call(L, **bad) == bdla.ERR_SHAPE, bad
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(base=0.5), dict(base=float("inf"))):
        assert _call(L, **bad) == bdla.ERR_RANGE, bad
    assert _call(L, page=65537) == bdla.ERR_UNSUPPORTED
    assert _call(L, n_pages=1 << 28) == _call(L, max_pages=1 << 28) == bdla.ERR_TOO_LARGE
    for less in (dict(ws=None), dict(ws_bytes=255), dict(ws=P + 8)):
        assert _call(L, **less) == bdla.ERR_WORKSPACE
        assert _call(L, q=None, wq=None, qn=None, **less) == bdla.ERR_WORKSPACE   # keys and values alone: the rest is in order


def test_refusals_of_packed_tokens(L):
    packed = dict(dims=(1, 5, 8, 2, 128), cu=P, n_docs=3)
    assert _call(L, **packed) == bdla.ERR_UNSUPPORTED          # rows and counts
    assert _call(L, rows=None, **packed) == bdla.ERR_UNSUPPORTED
    assert _call(L, counts=None, **packed) == bdla.ERR_UNSUPPORTED
    assert _call(L, rows=None, counts=None, ws=None, **packed) == bdla.ERR_WORKSPACE
    for bad in (dict(dims=(2, 5, 8, 2, 128)), dict(n_docs=0)):
        assert _call(L, rows=None, counts=None, **{**packed, **bad}) == bdla.ERR_SHAPE
    assert _call(L, rows=None, counts=None, **{**packed, "n_docs": 65536}) == bdla.ERR_UNSUPPORTED
