"""The smallest and oddest arguments of the softmax layer's entry points, as far as they need no GPU."""
import os
import subprocess
import sys

import pytest
import torch

from chunked_linear_attention_bounded_gb300 import bdla
from chunked_linear_attention_bounded_gb300.build import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    build()
    return bdla.lib()


def test_workspace_of_no_new_tokens_is_an_answer(L):
    """0 bytes, as for all sizes that the call refuses, and not the end of the process (a child, so that such an end
    would fail this test alone); the other operators take no tokens."""
    code = ("from chunked_linear_attention_bounded_gb300 import bdla\n"
            "size = bdla.lib().bdla_workspace_bytes_attn\n"
            "print([size(op, bdla.AttnDims(B, 0, 8, 2, d), 0, keys) for op in range(5) for B in (1, 2) for d in (64, 128)"
            " for keys in (0, 1024)])")
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert run.returncode == 0, (run.returncode, run.stderr)
    sizes = eval(run.stdout)
    assert all(n >= 256 for n in sizes[:32]) and sizes[32:] == [0] * 8


def test_refused_sizes_raise_what_the_call_says(L):
    """Where the workspace query has no answer the call is asked, without a workspace: it refuses before a launch."""
    asked = []

    def call(p, n):
        asked.append((p, n))
        return bdla.ERR_SHAPE

    with pytest.raises(bdla.BdlaError) as e:
        bdla._with_ws("bdla_attn_cached", bdla.ATTN_CACHED, bdla.AttnDims(2, 0, 8, 2, 128), 0, 1024, None, "cpu", None, call)
    assert e.value.status == bdla.ERR_SHAPE and asked == [(None, 0)]
    cache = bdla.CacheArgs(1 << 20, 1 << 20, 1 << 20, 1 << 20, 4, 16, 2)
    for T, status in ((0, bdla.ERR_SHAPE), (65, bdla.ERR_UNSUPPORTED)):
        assert L.bdla_attn_cached(1 << 20, cache, None, 0.1, 1 << 20, 1 << 20, bdla.AttnDims(2, T, 8, 2, 128), None, 0,
                                  None) == status


def test_strides_of_a_projections_views():
    """Token and head strides of [B, T, H, d]; a stride along an axis without a second entry says nothing."""
    f = lambda shape, strides: bdla._token_strides(shape, strides, "q")
    assert f((2, 5, 3, 64), (5 * 448, 448, 64, 1)) == (448, 64)
    assert f((3, 1, 3, 64), (448, 7, 64, 1)) == (448, 64)        # one token a row
    assert f((2, 5, 1, 64), (5 * 448, 448, 3, 1)) == (448, 64)   # one head
    assert f((1, 5, 2, 64), (9, 448, 64, 1)) == (448, 64)        # one row
    assert f((1, 1, 2, 64), (9, 5, 64, 1)) == (128, 64)          # one token
    for B in (1, 2):                                             # no token: torch's own strides, and others
        empty = torch.empty((B, 0, 4, 64))
        assert f(tuple(empty.shape), empty.stride()) == (256, 64)
        assert f((B, 0, 4, 64), (3, 5, 64, 1)) == (256, 64)
    with pytest.raises(ValueError, match="batch rows"):
        f((2, 5, 3, 64), (6 * 448, 448, 64, 1))
    with pytest.raises(ValueError, match="features"):
        f((2, 5, 3, 64), (5 * 448, 448, 1, 64))


def test_a_workspace_keeps_its_record_as_it_grows(monkeypatch):
    """The status word survives growth (on any device), the scratch behind it starts at zero."""
    monkeypatch.setattr(bdla, "_capturing", lambda: False)
    ws = bdla.Workspace(256, "cpu")
    ws.buf[:256] = torch.arange(256, dtype=torch.uint8)
    assert ws.ensure(200) is ws and ws.nbytes == 256
    ws.ensure(5000)
    assert ws.nbytes == ws.buf.numel() == 5000 and not ws.held
    assert torch.equal(ws.buf[:256], torch.arange(256, dtype=torch.uint8)) and not bool(ws.buf[256:].any())


def test_growing_in_a_capture_leaves_the_record_where_it_is(monkeypatch):
    """Nothing is copied, which the graph would repeat; the outgrown record is still read, and first."""
    monkeypatch.setattr(bdla, "_capturing", lambda: True)
    ws = bdla.Workspace(256, "cpu")
    first = ws.buf
    first[0] = 10
    ws.ensure(1000)
    assert not bool(ws.buf.any()) and ws.held == [first]
    asked = []
    monkeypatch.setattr(bdla, "_stream_handle", lambda s: None)
    monkeypatch.setattr(bdla, "lib", lambda: type("L", (), {
        "bdla_read_device_status": staticmethod(lambda p, s: asked.append(p.value) or (10 if p.value == first.data_ptr() else 0))}))
    assert ws.read_device_status() == bdla.ERR_DEVICE
    assert asked == [first.data_ptr(), ws.buf.data_ptr()]


def test_buffers_that_a_graph_may_hold_outlive_growth(monkeypatch):
    capturing = [True]
    monkeypatch.setattr(bdla, "_capturing", lambda: capturing[0])
    ws = bdla.Workspace(300, "cpu")
    first = ws.buf
    calls = []

    def call(p, n):
        calls.append(n)
        return bdla.OK if n >= 300 else bdla.ERR_WORKSPACE

    bdla._with_ws("x", bdla.ATTN_FWD, bdla.AttnDims(1, 4, 4, 2, 64), 0, 0, ws, torch.device("cpu"), None, call)   # captured
    assert calls == [300] and ws.in_graph
    capturing[0] = False
    second = ws.ensure(1000).buf       # grown outside, twice
    ws.ensure(2000)
    assert [b.data_ptr() for b in ws.held] == [first.data_ptr(), second.data_ptr()]
    ws = bdla.Workspace(300, "cpu")    # no capture: the old buffers go
    bdla._with_ws("x", bdla.ATTN_FWD, bdla.AttnDims(1, 4, 4, 2, 64), 0, 0, ws, torch.device("cpu"), None, call)
    ws.ensure(1000)
    assert not ws.in_graph and not ws.held


def test_tensors_off_the_current_device_are_refused(monkeypatch):
    class OnSecond:
        device = torch.device("cuda", 1)
        get_device = staticmethod(lambda: 1)

    monkeypatch.setattr(bdla, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device is cuda:0"):
        bdla._here(OnSecond, "q")
    monkeypatch.setattr(bdla, "_current_device", lambda: 1)
    bdla._here(OnSecond, "q")


def test_a_workspace_on_another_device_is_refused():
    ws = bdla.Workspace(1000, "cpu")
    launch = lambda p, n: pytest.fail("reached the library")
    with pytest.raises(ValueError, match="ws is on cpu"):
        bdla._with_ws("x", bdla.ATTN_FWD, bdla.AttnDims(1, 4, 4, 2, 64), 0, 0, ws, torch.device("cuda", 0), None, launch)
    with pytest.raises(ValueError, match="ws is on cpu"):
        bdla._workspace(256, torch.device("cuda", 0), ws, None)
