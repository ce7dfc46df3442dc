"""The smallest and oddest arguments of the softmax layer's calls on a GPU."""
import pytest
import torch

from chunked_linear_attention_bounded_gb300 import bdla

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("nbytes", [None, 256, 1 << 20])
def test_attn_cached_refuses_no_new_tokens(nbytes):
    q = torch.empty((2, 0, 8, 128), dtype=BF16, device="cuda")
    kc = torch.zeros((4, 16, 2, 128), dtype=BF16, device="cuda")
    table = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = None if nbytes is None else bdla.Workspace(nbytes, "cuda")
    with pytest.raises(bdla.BdlaError) as e:
        bdla.attn_cached(q, kc, kc, table, lens, ws=ws)
    assert e.value.status == bdla.ERR_SHAPE


@pytest.mark.parametrize("B", [1, 2])
def test_norm_of_rows_without_tokens(B):
    q, k = torch.empty((B, 0, 4, 64), dtype=BF16, device="cuda"), torch.empty((B, 0, 2, 64), dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    qn, kn = bdla.qk_norm(q, k, w, w)
    assert qn.shape == q.shape and kn.shape == k.shape
    dq, dk, dwq, dwk = bdla.qk_norm_bwd(q, k, w, w, q, k)
    assert dq.shape == q.shape and dk.shape == k.shape
    assert float(dwq.abs().sum() + dwk.abs().sum()) == 0.0


def test_norm_of_one_token_whatever_its_token_stride_says():
    """A step of one sequence: the strides of its single row and token mean nothing."""
    flat = torch.randn(6 * 64, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(BF16)
    q, k = torch.as_strided(flat, (1, 1, 4, 64), (3, 5, 64, 1)), torch.as_strided(flat, (1, 1, 2, 64), (7, 1, 64, 1), 256)
    w = torch.linspace(0.5, 1.5, 64, device="cuda")
    got = bdla.qk_norm(q, k, w, w)
    want = bdla.qk_norm(q.clone(memory_format=torch.contiguous_format), k.clone(memory_format=torch.contiguous_format), w, w)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def _cache(page=16, pages=4, Hk=2, d=64):
    kc = torch.randn((pages, page, Hk, d), generator=torch.Generator("cuda").manual_seed(2), device="cuda").to(BF16)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    return kc, kc.clone(), table, torch.tensor([pages * page - 8], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("on_side_stream", [False, True])
def test_an_error_recorded_before_the_workspace_grows_is_still_read(on_side_stream):
    """A bad page seen by an append, then attention that needs partial sums in the same workspace."""
    kc, vc, table, lens = _cache(pages=400)
    stream = torch.cuda.Stream() if on_side_stream else None
    k, q = torch.zeros((1, 1, 2, 64), dtype=BF16, device="cuda"), torch.zeros((1, 1, 4, 64), dtype=BF16, device="cuda")
    bad = table.clone()
    bad[0, -1] = 400
    ws = bdla.Workspace(256, "cuda")
    torch.cuda.synchronize()
    bdla.cache_append(k, k, kc, vc, bad, lens, ws=ws, stream=stream)
    assert ws.nbytes == 256
    bdla.attn_cached(q, kc, vc, table, lens, ws=ws, stream=stream)
    assert ws.nbytes > 256   # it grew
    assert ws.read_device_status(stream) == bdla.ERR_DEVICE
    assert ws.read_device_status(stream) == bdla.OK


def test_a_workspace_grows_on_the_stream_of_the_call():
    """A call on an idle stream while the current one is busy: were the new buffer cleared on the busy one, the clearing
    would come after the call and take what it recorded with it.  Linear attention and softmax attention."""
    g = torch.Generator("cuda").manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    q, k, v, a = rn(1, 300, 2, 64).to(BF16), rn(1, 300, 2, 64).to(BF16), rn(1, 300, 2, 64).to(BF16), rn(1, 300, 2)
    bad = torch.tensor([0, 200, 100, 300], dtype=torch.int32, device="cuda")   # reported, and left out
    o, lse = torch.zeros_like(q), torch.zeros((2, 300), device="cuda")
    busy = torch.ones((4096, 4096), device="cuda")
    side = torch.cuda.Stream()
    for call in (lambda ws: bdla.fwd(q, k, v, a, cu_seqlens=bad, ws=ws, stream=side),
                 lambda ws: bdla.attn_bwd(q, k, v, o, lse, q, cu_seqlens=bad, ws=ws, stream=side)):
        ws = bdla.Workspace(256, "cuda")
        torch.cuda.synchronize()
        for _ in range(20):
            torch.mm(busy, busy)
        kept = call(ws)   # its outputs live until everything is done
        assert ws.nbytes > 256
        torch.cuda.synchronize()
        assert ws.read_device_status(side) == bdla.ERR_DEVICE
        del kept


def test_a_graph_replays_on_its_buffer_after_the_workspace_has_grown():
    """A decode step captured with a workspace that a larger call outgrows later: the replay's partial sums and record
    go to the buffer that the graph knows, which nothing else has been given meanwhile."""
    kc, vc, table, lens = _cache(pages=400)
    q = torch.randn((1, 1, 4, 64), generator=torch.Generator("cuda").manual_seed(5), device="cuda").to(BF16)
    want = bdla.attn_cached(q, kc, vc, table, lens)
    need = bdla.lib().bdla_workspace_bytes_attn(bdla.ATTN_CACHED, bdla.AttnDims(1, 1, 4, 2, 64), 0, 6400)
    ws = bdla.Workspace(need, "cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = bdla.attn_cached(q, kc, vc, table, lens, ws=ws)
    assert ws.nbytes == need
    ws.ensure(4 * need)
    others = [torch.full((need,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]   # whoever asks for such a size
    for x in got:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert all(bool((x == 7).all()) for x in others)
    assert ws.read_device_status() == bdla.OK
    table[0, 0] = 400
    graph.replay()
    assert ws.read_device_status() == bdla.ERR_DEVICE   # the replay's own record
    assert ws.read_device_status() == bdla.OK


def _calls():
    """Every public call with small right arguments, as (name, f(ws))."""
    rn = lambda *s: torch.randn(s, generator=torch.Generator("cuda").manual_seed(7), device="cuda")
    q, k, a = rn(1, 20, 4, 64).to(BF16), rn(1, 20, 2, 64).to(BF16), rn(1, 20, 4)
    w, lse = torch.ones(64, device="cuda"), torch.zeros((4, 20), device="cuda")
    kc, vc, table, lens = _cache()
    lens = lens - 20
    state, av, beta = torch.zeros((1, 4, 64, 64), device="cuda"), rn(1, 20, 4, 64), torch.sigmoid(a)
    q1, a1 = q[:, 0].contiguous(), a[:, 0].contiguous()
    return [("qk_norm", lambda ws: bdla.qk_norm(q, k, w, w)),
            ("qk_norm_bwd", lambda ws: bdla.qk_norm_bwd(q, k, w, w, q, k, ws=ws)),
            ("attn_fwd", lambda ws: bdla.attn_fwd(q, k, k, ws=ws)),
            ("attn_bwd", lambda ws: bdla.attn_bwd(q, k, k, q, lse, q, ws=ws)),
            ("cache_append", lambda ws: bdla.cache_append(k, k, kc, vc, table, lens, ws=ws)),
            ("attn_cached", lambda ws: bdla.attn_cached(q, kc, vc, table, lens, ws=ws)),
            ("fwd", lambda ws: bdla.fwd(q, q, q, a, ws=ws)),
            ("bwd", lambda ws: bdla.bwd(q, q, q, a, q, ws=ws)),
            ("decode", lambda ws: bdla.decode(q1, q1, q1, a1, state)),
            ("decay", lambda ws: bdla.decay(a, ws=ws)),
            ("fwd_vec", lambda ws: bdla.fwd_vec(q, q, q, av, ws=ws)),
            ("fwd_delta", lambda ws: bdla.fwd_delta(q, q, q, a, beta, ws=ws))]


def test_calls_off_the_current_device_or_with_a_workspace_from_elsewhere_are_refused(monkeypatch):
    calls = _calls()
    elsewhere = bdla.Workspace(1 << 20, "cpu")
    for name, f in calls:
        f(None)
        f(bdla.Workspace(256, "cuda"))
        if name not in ("qk_norm", "decode"):
            with pytest.raises(ValueError, match="ws is on cpu"):
                f(elsewhere)
    torch.cuda.synchronize()
    monkeypatch.setattr(bdla, "_current_device", lambda: 1)
    for name, f in calls:
        with pytest.raises(ValueError, match="current device is cuda:1"):
            f(None)


def test_cache_arguments_are_refused_by_name():
    kc, vc, table, lens = _cache()
    q = torch.zeros((1, 1, 4, 64), dtype=BF16, device="cuda")
    for change, message in ((dict(pages=table.repeat(2, 1)), "pages must be"), (dict(pages=table[0]), "pages must have 2"),
                            (dict(pages=table.long()), "pages must be torch.int32"), (dict(lens=lens.repeat(2)), "lens must be"),
                            (dict(vcache=vc[:2]), "vcache must be"), (dict(kcache=kc.float()), "kcache must be torch.bfloat16"),
                            (dict(kcache=kc.transpose(0, 1)), "kcache must be contiguous"), (dict(pages=table.cpu()), "CUDA")):
        args = dict(kcache=kc, vcache=vc, pages=table, lens=lens)
        args.update(change)
        with pytest.raises(ValueError, match=message):
            bdla.attn_cached(q, **args)
        with pytest.raises(ValueError, match=message):
            bdla.cache_append(q[:, :, :2].contiguous(), q[:, :, :2].contiguous(), **args)
