"""The hybrid example: its softmax layer's gradients against automatic differentiation of the whole layer in 64 bits,
and its serving path against whole-prompt attention."""
import os
import sys

import pytest
import torch

import _attn_ref as ref
from _parity import REL_L2

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import hybrid_layer as ex  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64


def _layer64(x, w, R, eps):
    return torch.einsum("btij,bthj->bthi", R, x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w)


def test_softmax_layer_gradient_through_norm_rotation_and_attention():
    """The chain of kernels, each with its own bf16 outputs, stays within the parity bar of the library."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    layer = ex.Layer(Hq=4, Hk=2)
    lens = (130, 1, 169)
    cu = torch.tensor([0, 130, 131, 300], dtype=torch.int32, device="cuda")
    qkv, a = rn(1, 300, 8, 128).to(BF16), rn(1, 300, 4)
    dO = rn(1, 300, 4, 128).to(BF16)
    none = torch.zeros_like(dO)     # nothing upstream of the linear layer: its part of the gradients is zero
    o, _, grads = ex.train_step(layer, qkv, a, dO, none, cu)
    leaves = [x.to(F64).requires_grad_() for x in (qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:], layer.wq, layer.wk)]
    q, k, v, wq, wk = leaves
    R = ref.rotation(ref.positions(1, 300, cu, "cuda"), 128, 10000.0, 128, False)
    qn, kn = _layer64(q, wq, R, 1e-6), _layer64(k, wk, R, 1e-6)
    out, at = [], 0
    for n in lens:
        s = slice(at, at + n)
        kk, vv = (x[0, s].repeat_interleave(2, 1) for x in (kn, v))
        x = torch.einsum("ihd,jhd->hij", qn[0, s], kk) * 128 ** -0.5
        x = x.masked_fill(~torch.ones((n, n), dtype=torch.bool, device="cuda").tril(), -torch.inf)
        out.append(torch.einsum("hij,jhd->ihd", x.softmax(-1), vv))
        at += n
    want = torch.cat(out)[None]
    want.backward(dO.to(F64))
    near = lambda x, y: float((x.to(F64) - y).norm() / y.norm())
    # norm, attention and their gradients round in turn: each stage within its own bar
    assert near(o, want.detach()) <= REL_L2
    for n, x in zip(("q", "k", "v", "wq", "wk"), leaves):
        assert near(grads[n], x.grad) <= 2 * REL_L2, n


def test_serving_path_agrees_with_the_whole_prompt():
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF16)
    layer = ex.Layer(Hq=8, Hk=2)
    prompt, draft, then = rn(1, 333, 12, 128), rn(1, 6, 12, 128), rn(1, 1, 12, 128)
    tree = torch.tensor([[0b1, 0b11, 0b101, 0b1101, 0b10000, 0b110000]], dtype=torch.int64, device="cuda")
    depth = torch.tensor([[0, 1, 1, 2, 0, 1]], device="cuda")
    path = [0, 2, 3]
    o_prompt, o_draft, o_then = ex.serve(layer, prompt, draft, tree, depth, path, then)
    whole = torch.cat([prompt, draft[:, path], then], 1)
    qn, kn = ex.bdla.qk_norm(whole[:, :, :8], whole[:, :, 8:10], layer.wq, layer.wk)
    want = ref.attn(qn, kn, whole[:, :, 10:].contiguous(), 128 ** -0.5)["o"]
    ref.check("prompt", o_prompt, tuple(x[:, :333] for x in want))
    ref.check("accepted drafts", o_draft[:, path], tuple(x[:, 333:336] for x in want))
    ref.check("the token after", o_then, tuple(x[:, 336:] for x in want))


def test_example_runs():
    ex.main()
