"""attn_bwd where key tiles are many: one CTA walks the queries of every head of its group, and nothing is joined."""
import pytest
import torch

import _attn_ref as ref
from chunked_linear_attention_bounded_gb300 import bdla

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

GROUPED = [
    # B, T, lens, Hq, Hk, d: odd documents whose last tiles are ragged in the middle of a CTA's walk over the heads
    (1, 2600, (1001, 1, 1598), 16, 8, 128),
    (1, 2600, (129, 0, 127, 2344), 24, 8, 64),
    (3, 901, None, 20, 10, 64),
    (2, 1279, None, 64, 8, 128),
]


def _inputs(case, seed=0):
    B, T, lens, Hq, Hk, d = case
    g = torch.Generator("cuda").manual_seed(T + Hq + seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF16)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda") if lens else None
    # without partial sums a workspace holds the status and delta alone
    need = bdla.lib().bdla_workspace_bytes_attn(bdla.ATTN_BWD, bdla.AttnDims(B, T, Hq, Hk, d), len(lens or ()), 0)
    assert need == 256 + (B * T * Hq * 4 + 255) // 256 * 256, "not the path this test is about"
    return rn(B, T, Hq, d) * 2, rn(B, T, Hk, d), rn(B, T, Hk, d), rn(B, T, Hq, d), cu


@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "-".join(str(x) for x in c))
def test_gradient_over_the_heads_of_a_group(case):
    q, k, v, dO, cu = _inputs(case)
    want = ref.attn(q, k, v, case[5] ** -0.5, cu, dO)
    o, lse = want["o"][0].to(BF16), want["lse"][0].float()
    ws = bdla.Workspace(256, "cuda")
    got = bdla.attn_bwd(q, k, v, o, lse, dO, cu_seqlens=cu, ws=ws)
    assert ws.read_device_status() == bdla.OK
    for n, x in zip(("dq", "dk", "dv"), got):
        ref.check(n, x, want[n])
    again = bdla.attn_bwd(q, k, v, o, lse, dO, cu_seqlens=cu, ws=ws)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


def test_each_query_head_adds_its_own_part():
    """The gradients of k and v are the sums of those that each query head alone gives: no head is left out, taken twice
    or taken for another, which sums over like heads would hide."""
    case = GROUPED[0]
    q, k, v, dO, cu = _inputs(case, seed=1)
    scale, G = case[5] ** -0.5, case[3] // case[4]
    o, lse = bdla.attn_fwd(q, k, v, cu_seqlens=cu)
    for head in range(G):
        one = torch.zeros_like(dO)
        one[:, :, head::G] = dO[:, :, head::G]
        _, dk, dv = bdla.attn_bwd(q, k, v, o, lse, one, cu_seqlens=cu)
        want = ref.attn(q[:, :, head::G], k, v, scale, cu, dO[:, :, head::G])
        ref.check(f"dk of head {head}", dk, want["dk"])
        ref.check(f"dv of head {head}", dv, want["dv"])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("d", [64, 128])
def test_documents_do_not_reach_each_other_through_a_group(bad, d):
    """A document of infinities or NaN between two whose last tiles end inside it changes nothing in them."""
    lens = (1100, 300, 1201)
    q, k, v, dO, cu = _inputs((1, sum(lens), lens, 24, 8, d), seed=2)
    o, lse = bdla.attn_fwd(q, k, v, cu_seqlens=cu)
    clean = bdla.attn_bwd(q, k, v, o, lse, dO, cu_seqlens=cu)
    for x in (q, k, v, dO):
        x[:, 1100:1400] = bad
    o2, lse2 = bdla.attn_fwd(q, k, v, cu_seqlens=cu)
    o3 = o.clone()
    o3[:, 1100:1400] = bad
    dirty = bdla.attn_bwd(q, k, v, o3, lse2, dO, cu_seqlens=cu)
    for x, y in [(o, o2)] + list(zip(clean, dirty)):
        assert torch.equal(x[:, :1100], y[:, :1100]) and torch.equal(x[:, 1400:], y[:, 1400:])
    assert torch.equal(lse[:, :1100], lse2[:, :1100]) and torch.equal(lse[:, 1400:], lse2[:, 1400:])
