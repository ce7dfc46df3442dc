"""The linear half of the hybrid example's training step against the 64-bit oracle, alone and beside the softmax half."""
import os
import sys

import pytest
import torch

import oracle
from _parity import REL_L2

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import hybrid_layer as ex  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
CU, Hq, Hk, d = [0, 130, 131, 300], 4, 2, 128


def _inputs(seed):
    g = torch.Generator("cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    return (rn(1, 300, Hq + 2 * Hk, d).to(BF16), rn(1, 300, Hq), rn(1, 300, Hq, d).to(BF16), rn(1, 300, Hq, d).to(BF16),
            torch.tensor(CU, dtype=torch.int32, device="cuda"))


def _near(x, y):
    return float((x.to(F64).cpu() - y).norm() / y.norm())


def _linear64(qkv, a, dO):
    """Output and gradients of the linear layer: unit keys and queries, keys and values shared by their group."""
    q, k, v = (x.clone().requires_grad_() for x in qkv.to(F64).cpu().split([Hq, Hk, Hk], 2))
    unit = lambda x: x / (x * x).sum(-1, keepdim=True).add(1e-12 * d).sqrt()
    shared = [unit(q)[0], unit(k)[0].repeat_interleave(Hq // Hk, 1), v[0].repeat_interleave(Hq // Hk, 1)]
    args = [x.detach().numpy() for x in shared] + [a[0].to(F64).cpu().numpy()]
    o, _ = oracle.fwd(*args, cu_seqlens=CU)
    *grads, da, _ = oracle.bwd(*args, dO[0].to(F64).cpu().numpy(), cu_seqlens=CU)
    torch.autograd.backward(shared, [torch.from_numpy(x) for x in grads])
    return torch.from_numpy(o)[None], dict(q=q.grad, k=k.grad, v=v.grad, a=torch.from_numpy(da)[None])


def test_linear_layer_and_its_gradients():
    """Norm, linear attention, its gradient and the norm's gradient, each with its own roundings, stay within the
    library's bar a stage: two for the output, and for the gradients."""
    qkv, a, dO, dO_linear, cu = _inputs(4)
    layer = ex.Layer(Hq=Hq, Hk=Hk)
    _, ol, grads = ex.train_step(layer, qkv, a, torch.zeros_like(dO), dO_linear, cu)
    want_o, want = _linear64(qkv, a, dO_linear)
    assert _near(ol, want_o) <= 2 * REL_L2
    for n, x in want.items():
        assert _near(grads[n], x) <= 2 * REL_L2, n
    assert float(grads["wq"].abs().max()) == float(grads["wk"].abs().max()) == 0.0   # the linear norm's are not learned
    for ws in layer.ws.values():
        assert ws.read_device_status() == ex.bdla.OK


def test_the_two_layers_gradients_add_up():
    """The step with both upstream gradients gives the sum of the steps with one: the bf16 parts are added in bf16, one
    more rounding of half a step of the sum."""
    qkv, a, dO, dO_linear, cu = _inputs(5)
    layer = ex.Layer(Hq=Hq, Hk=Hk)
    none = torch.zeros_like(dO)
    o, ol, both = ex.train_step(layer, qkv, a, dO, dO_linear, cu)
    o1, _, soft = ex.train_step(layer, qkv, a, dO, none, cu)
    _, ol2, lin = ex.train_step(layer, qkv, a, none, dO_linear, cu)
    assert torch.equal(o, o1) and torch.equal(ol, ol2)
    for n in ("q", "k", "v", "a"):
        assert _near(both[n], (soft[n].to(F64) + lin[n].to(F64)).cpu()) <= 2.0 ** -8, n
        assert float(lin[n].abs().max()) > 0 and (n == "a") == (float(soft[n].abs().max()) == 0), n
    for n in ("wq", "wk"):
        assert torch.equal(both[n], soft[n])
