"""Arguments that bdla_attn_shared refuses on the host, before any launch (fake pointers are never read)."""
import pytest

from chunked_linear_attention_bounded_gb300 import bdla
from chunked_linear_attention_bounded_gb300.build import build

P = 1 << 20


@pytest.fixture(scope="module")
def L():
    build()
    return bdla.lib()


def _call(L, dims=(3, 1, 8, 2, 128), n=2, scale=0.1, q=P, kc=P, vc=P, pages=P, lens=P, cu=P, shared=P, tree=None, o=P, lse=P,
          ws=P, ws_bytes=1 << 40, n_pages=9, page=16, max_pages=4):
    return L.bdla_attn_shared(q, bdla.CacheArgs(kc, vc, pages, lens, n_pages, page, max_pages), cu, shared, n, tree, scale, o, lse,
                              bdla.AttnDims(*dims), ws, ws_bytes, None)


def test_refusals(L):
    for dims, want in (((0, 1, 8, 2, 128), bdla.ERR_SHAPE), ((3, 0, 8, 2, 128), bdla.ERR_SHAPE), ((3, 1, 8, 3, 128), bdla.ERR_SHAPE),
                       ((3, 65, 8, 2, 128), bdla.ERR_UNSUPPORTED), ((3, 1, 8, 2, 96), bdla.ERR_UNSUPPORTED),
                       ((65536, 1, 8, 2, 128), bdla.ERR_UNSUPPORTED), ((65535, 64, 1024, 1, 64), bdla.ERR_TOO_LARGE),
                       ((65535, 64, 256, 1, 64), bdla.ERR_TOO_LARGE)):
        assert _call(L, dims=dims) == want, dims
    assert _call(L, n=0) == _call(L, n=-1) == bdla.ERR_SHAPE
    assert _call(L, n=65536) == bdla.ERR_UNSUPPORTED
    for x in ("q", "kc", "vc", "pages", "lens", "cu", "shared", "o", "lse"):
        assert _call(L, **{x: None}) == bdla.ERR_NULL, x
    for x in ("q", "kc", "vc", "o"):
        assert _call(L, **{x: P + 8}) == bdla.ERR_ALIGN, x
    for x in ("cu", "shared", "lse", "tree"):
        assert _call(L, **{x: P + 2}) == bdla.ERR_ALIGN, x
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert _call(L, scale=s) == bdla.ERR_RANGE
    assert _call(L, page=65537) == bdla.ERR_UNSUPPORTED
    need = L.bdla_workspace_bytes_attn(bdla.ATTN_SHARED, bdla.AttnDims(3, 1, 8, 2, 128), 2, 64)
    assert need > 256
    for less in (dict(ws=None), dict(ws_bytes=need - 1), dict(ws=P + 8)):
        assert _call(L, **less) == bdla.ERR_WORKSPACE


def test_the_threshold_is_a_setting(L):
    for n in (0, 1 << 40, -1):
        assert L.bdla_set_share_least(n) == bdla.OK


def test_workspace_sizes(L):
    size = lambda dims, n, keys: L.bdla_workspace_bytes_attn(bdla.ATTN_SHARED, bdla.AttnDims(*dims), n, keys)
    d = (256, 1, 32, 8, 128)
    assert size(d, 1, 1 << 16) == size(d, 1, 1 << 20) > 256        # by the rows, not by the table's width
    assert size(d, 1, 1 << 16) < 200 << 20
    for bad in (((256, 0, 32, 8, 128), 1, 64), ((256, 65, 32, 8, 128), 1, 64), (d, 0, 64), (d, 65536, 64), (d, 1, -1),
                ((256, 1, 30, 8, 128), 1, 64), ((65535, 64, 256, 1, 64), 1, 64)):
        assert size(*bad) == 0, bad
