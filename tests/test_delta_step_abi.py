"""Arguments that bdla_decode_delta refuses on the host, before any launch (fake pointers are never read)."""
import ctypes

import pytest

from chunked_linear_attention_bounded_gb300 import bdla
from chunked_linear_attention_bounded_gb300.build import build

P = 1 << 20


@pytest.fixture(scope="module")
def L():
    build()
    return bdla.lib()


def _call(L, dims=(4, 1, 2, 128, 128), b=-5.0, mode=0, n_slots=4, o_dtype=0, ws_bytes=1 << 20, **p):
    a = dict.fromkeys(("q", "k", "v", "a", "beta", "state", "slots", "counts", "o", "ws"), P)
    a.update(p)
    return L.bdla_decode_delta(a["q"], a["k"], a["v"], a["a"], a["beta"], b, a["state"], a["slots"], n_slots, a["counts"],
                               a["o"], o_dtype, bdla.Dims(*dims), mode, a["ws"], ws_bytes, None)


def test_refusals(L):
    for dims, want in (((0, 1, 2, 128, 128), bdla.ERR_SHAPE), ((4, 0, 2, 128, 128), bdla.ERR_SHAPE),
                       ((4, -1, 2, 128, 128), bdla.ERR_SHAPE), ((4, 1, 0, 128, 128), bdla.ERR_SHAPE),
                       ((4, 1, 2, 96, 128), bdla.ERR_UNSUPPORTED), ((4, 1, 2, 128, 256), bdla.ERR_UNSUPPORTED),
                       ((65536, 1, 2, 128, 128), bdla.ERR_UNSUPPORTED), ((65535, 1, 1 << 20, 128, 128), bdla.ERR_TOO_LARGE),
                       ((65535, 1 << 16, 1, 64, 64), bdla.ERR_TOO_LARGE)):
        assert _call(L, dims=dims) == want, dims
    for b in (0.5, float("nan"), -5.5):
        assert _call(L, b=b) == bdla.ERR_RANGE
    assert _call(L, mode=2) == bdla.ERR_UNSUPPORTED
    assert _call(L, n_slots=-1) == bdla.ERR_SHAPE
    assert _call(L, o_dtype=2) == bdla.ERR_DTYPE
    for x in ("q", "k", "v", "a", "beta", "state", "o"):
        assert _call(L, **{x: None}) == bdla.ERR_NULL, x
        assert _call(L, **{x: P + 4}) == bdla.ERR_ALIGN, x
    for x in ("slots", "counts"):
        assert _call(L, **{x: P + 2}) == bdla.ERR_ALIGN, x
    # the status word is needed where the device may have something to say
    for less in (dict(ws=None), dict(ws_bytes=255), dict(ws=P + 8)):
        assert _call(L, **less) == bdla.ERR_WORKSPACE
        assert _call(L, slots=None, **less) == _call(L, counts=None, **less) == bdla.ERR_WORKSPACE


def test_the_grid_is_a_limit_of_its_own(L):
    """A CTA takes 16 columns of a state of 128 rows and 32 of one of 64; 65535 x 8192 states of 128 columns lie between
    the two."""
    assert _call(L, dims=(65535, 1, 8192, 128, 128)) == bdla.ERR_TOO_LARGE
    assert _call(L, dims=(65535, 1, 8192, 128, 64), ws=None) == bdla.ERR_WORKSPACE   # the last check before the launch
    assert _call(L, dims=(65535, 1, 8192, 64, 128), ws=None) == bdla.ERR_WORKSPACE
    assert _call(L, dims=(65535, 1, 8193, 64, 128)) == bdla.ERR_TOO_LARGE
