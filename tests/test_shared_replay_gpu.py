"""Attention over shared pages in a serving loop: everything that a call reads is rewritten in place between replays of one
captured call, with nothing but stream order between the writes and the replay."""
import pytest
import torch

import _attn_ref as ref
from chunked_linear_attention_bounded_gb300 import bdla
from test_shared_gpu import _batch, _call

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _trees(B, T, g):
    bits = torch.rand((B, T, T), generator=g, device="cuda") < 0.5
    return (bits.long() << torch.arange(T, device="cuda")).sum(2)


# new tokens, query heads a key head, and what takes the sequences' own positions beside the tensor cores' shared ones
@pytest.mark.parametrize("T,Hq,page", [(1, 8, 16), (5, 8, 16), (1, 8, 24), (12, 8, 16)],
                         ids=["a warp a piece", "four warps a piece", "pages without TMA", "the tensor cores too"])
@pytest.mark.parametrize("tree", [False, True])
def test_a_replay_reads_what_was_written_last(T, Hq, page, tree):
    bdla.set_share_least(0)
    try:
        x = _batch([(20, 25), (6, 9)], 3, [40, 5, 300], T, Hq, 2, 128, page, tree=tree)
        ws = bdla.Workspace(1 << 27, "cuda")
        _call(x, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, lse = _call(x, ws)
    finally:
        bdla.set_share_least(-1)
    g = torch.Generator("cuda").manual_seed(5)
    n, B = x["kc"].shape[0], x["table"].shape[0]
    seen = []
    shrink = torch.tensor([0, 3, 17, 0, 2], dtype=I32, device="cuda")
    for i in range(5):
        to = torch.randperm(n, generator=g, device="cuda").to(I32)   # page p moves to place to[p], with new contents
        x["table"].copy_(torch.where(x["table"] >= 0, to[x["table"].clamp(min=0).long()], x["table"]))
        for c in (x["kc"], x["vc"]):
            new = torch.randn(c.shape, generator=g, device="cuda").to(c.dtype)
            c.copy_(torch.empty_like(c).index_copy_(0, to.long(), torch.where(c.isnan(), c, new)))
        x["q"].copy_(torch.randn(x["q"].shape, generator=g, device="cuda"))
        x["lens"].sub_(shrink[i]).clamp_(min=0)
        if tree:
            x["tree"].copy_(_trees(B, T, g))
        if i == 3:
            x["cu"].copy_(torch.tensor([2, 20, 26], dtype=I32))
            x["shared"].sub_(11)
        o.fill_(float("nan")), lse.fill_(float("nan"))
        graph.replay()
        seen.append({k: v.clone() for k, v in x.items() if v is not None} | dict(o=o.clone(), lse=lse.clone()))
    assert ws.read_device_status() == bdla.OK
    for y in seen:
        want_o, want_l = ref.cached(y["q"], y["kc"], y["vc"], y["table"], y["lens"].tolist(),
                                    y["tree"].cpu() if tree else None, 128 ** -0.5)
        ref.check("o", y["o"], want_o)
        ref.check("lse", y["lse"], want_l)
