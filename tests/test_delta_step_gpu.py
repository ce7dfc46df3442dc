"""Recurrent steps of the gated delta rule against the 64-bit oracle, and what slots and counts say about states."""
import numpy as np
import pytest
import torch

import oracle
from chunked_linear_attention_bounded_gb300 import bdla

from _parity import assert_close

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _tokens(B, T, H, dk, dv, seed=1, dev="cuda"):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)
    k = rn(B, T, H, dk)
    t = dict(q=(rn(B, T, H, dk) * dk ** -0.5).to(BF16), k=(k / k.norm(dim=-1, keepdim=True)).to(BF16),
             v=rn(B, T, H, dv).to(BF16), a=rn(B, T, H) * 1.5 - 2, beta=torch.rand((B, T, H), generator=g),
             state=rn(B, H, dk, dv) * 0.3)
    return {n: x.to(dev) for n, x in t.items()}


def _step(t, state, upto=None, first=0, **kw):
    part = {n: t[n][:, first:upto].contiguous() for n in ("q", "k", "v", "a", "beta")}
    return bdla.decode_delta(part["q"], part["k"], part["v"], part["a"], part["beta"], state, **kw)


def _oracle(t, mode):
    """o, final state and their tolerances.  Error of a column of S, by its norm: a token turns the error before it into
    at most as much (g <= 1, |I - beta k k^T| <= 1 with |k| <= 1), and adds the rounding of r (sums of dk products), of g
    (a few steps times |lambda| <= 8), of the update: at most (dk + 64) steps of fp32 of |S| + |v|."""
    f = lambda x: x.double().cpu().reshape(-1, *x.shape[2:]).numpy()
    B, T, H, dk = t["q"].shape
    cu = np.arange(B + 1) * T
    o, hT = oracle.fwd_delta(f(t["q"]), f(t["k"]), f(t["v"]), f(t["a"]), f(t["beta"]), -5.0, mode,
                             h0=t["state"].double().cpu().numpy(), cu_seqlens=cu)
    o = torch.from_numpy(o).view(B, T, H, -1)
    size = t["state"].double().cpu().norm(dim=2)[:, None] + t["v"].double().cpu().abs().cumsum(1)   # [B, T, H, dv]
    steps = torch.arange(1, T + 1).double()[None, :, None, None]
    err = 1.01 * steps * (dk + 64) * 2.0 ** -24 * size
    qn = t["q"].double().cpu().norm(dim=3, keepdim=True)
    return o, qn * (err + dk * 2.0 ** -24 * size), torch.from_numpy(hT), err[:, -1, :, None]


def _near(name, got, want, tol):
    far = (got.double().cpu() - want).abs() - tol
    assert bool((far <= 0).all()), f"{name}: {float(far.max())} outside"   # (a NaN is outside)


SIZES = [(1, 1, 1, 64, 64), (1, 1, 32, 128, 128), (5, 1, 3, 128, 64), (3, 7, 2, 64, 128), (2, 33, 5, 128, 128),
         (70, 2, 1, 64, 64), (1, 130, 2, 128, 64)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("mode", [bdla.BOUNDED, bdla.SOFTPLUS])
@pytest.mark.parametrize("o_dtype", [BF16, F32])
def test_steps_match_the_recurrence(size, mode, o_dtype):
    t = _tokens(*size)
    o, o_tol, hT, s_tol = _oracle(t, mode)
    state = t["state"].clone()
    got = _step(t, state, mode=mode, o_dtype=o_dtype)
    assert got.dtype == o_dtype and got.shape == o.shape
    _near("o", got, o, o_tol + (2.0 ** -8 * o.abs() if o_dtype == BF16 else 0))
    _near("state", state, hT, s_tol)


def test_tokens_together_or_one_call_each_give_the_same_bits():
    t = _tokens(4, 9, 3, 128, 128, seed=2)
    s1, s2 = t["state"].clone(), t["state"].clone()
    o1 = _step(t, s1)
    o2 = torch.cat([_step(t, s2, n + 1, n) for n in range(9)], 1)
    assert torch.equal(o1, o2) and torch.equal(s1, s2)


@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 64)])
def test_counts_say_which_state_is_left(dk, dv):
    B, T = 7, 6
    t = _tokens(B, T, 2, dk, dv, seed=3)
    want_o = _step(t, t["state"].clone())
    ends = [t["state"]]
    for n in range(1, T + 1):
        s = t["state"].clone()
        _step(t, s, n)
        ends.append(s)
    counts = torch.arange(B, dtype=torch.int32, device="cuda")
    state, ws = t["state"].clone(), bdla.Workspace(256, "cuda")
    o = _step(t, state, counts=counts, ws=ws)
    assert torch.equal(o, want_o)   # whatever is kept
    for b in range(B):
        assert torch.equal(state[b], ends[b][b]), b
    assert ws.read_device_status() == bdla.OK


def test_states_in_a_pool_and_unused_places():
    B, T, H, dk, dv = 9, 3, 4, 64, 64
    t = _tokens(B, T, H, dk, dv, seed=4)
    want_state = t["state"].clone()
    want_o = _step(t, want_state)
    pool = torch.randn((14, H, dk, dv), generator=torch.Generator().manual_seed(5)).cuda()
    before = pool.clone()
    slots = torch.tensor([13, 0, 7, -1, 2, 5, 4, -1, 9], dtype=torch.int32, device="cuda")
    used = slots >= 0
    pool[slots[used].long()] = t["state"][used]
    ws = bdla.Workspace(256, "cuda")
    o = _step(t, pool, slots=slots, ws=ws)
    assert torch.equal(o[used], want_o[used]) and not bool(o[~used].any())
    assert torch.equal(pool[slots[used].long()], want_state[used])
    rest = [i for i in range(14) if i not in slots.tolist()]
    assert torch.equal(pool[rest], before[rest])
    assert ws.read_device_status() == bdla.OK


def test_bad_slots_and_counts_are_recorded_and_touch_nothing():
    B, T, H, dk, dv = 80, 2, 2, 64, 128
    t = _tokens(B, T, H, dk, dv, seed=6)
    for bad, value in (("slots", B), ("slots", -2), ("slots", 3), ("slots", 2 ** 31 - 1), ("counts", -1), ("counts", T + 1)):
        slots = torch.arange(B, dtype=torch.int32, device="cuda")
        counts = torch.full((B,), T, dtype=torch.int32, device="cuda")
        (slots if bad == "slots" else counts)[60] = value   # slot 3 is sequence 3's
        state, ws = t["state"].clone(), bdla.Workspace(256, "cuda")
        o = _step(t, state, slots=slots, counts=counts, ws=ws)
        assert ws.read_device_status() == bdla.ERR_DEVICE, (bad, value)
        want = t["state"].clone()
        want_o = _step(t, want)
        want[60] = t["state"][60]
        if bad == "slots":
            want_o[60] = 0
        assert torch.equal(state, want) and torch.equal(o, want_o), (bad, value)
        assert ws.read_device_status() == bdla.OK


def test_an_empty_pool():
    t = _tokens(2, 1, 1, 64, 64)
    ws = bdla.Workspace(256, "cuda")
    o = _step(t, torch.empty((0, 1, 64, 64), device="cuda"), slots=torch.tensor([-1, -1], dtype=torch.int32, device="cuda"), ws=ws)
    assert not bool(o.any()) and ws.read_device_status() == bdla.OK
    o = _step(t, torch.empty((0, 1, 64, 64), device="cuda"), slots=torch.tensor([-1, 0], dtype=torch.int32, device="cuda"), ws=ws)
    assert not bool(o.any()) and ws.read_device_status() == bdla.ERR_DEVICE


def test_infinities_stay_with_their_sequence_head_and_column():
    t = _tokens(3, 2, 2, 128, 64, seed=7)
    want = t["state"].clone()
    want_o = _step(t, want)
    state = t["state"].clone()
    state[1, 0, 5, 40] = float("inf")
    t["v"][2, 0, 1, 3] = float("nan")
    o = _step(t, state)
    bad_s, bad_o = torch.zeros_like(state, dtype=torch.bool), torch.zeros_like(o, dtype=torch.bool)
    bad_s[1, 0, :, 40] = bad_s[2, 1, :, 3] = True
    bad_o[1, :, 0, 40] = bad_o[2, :, 1, 3] = True
    assert torch.equal(state[~bad_s], want[~bad_s]) and torch.equal(o[~bad_o], want_o[~bad_o])
    assert not bool(o[bad_o].isfinite().any())


def test_saturated_gates_and_write_strengths():
    """beta = 0 leaves the decayed state, a logit of -inf no decay, one of +inf the full bound; beta = 1 with a unit key
    stores the value (S^T k = v up to the key's own rounding)."""
    B, H, d = 2, 2, 64
    t = _tokens(B, 1, H, d, d, seed=8)
    t["beta"][0], t["beta"][1] = 0.0, 1.0
    t["a"][:, :, 0], t["a"][:, :, 1] = -1e4, 1e4
    t["k"][1] = 0
    t["k"][1, 0, 0, 17] = t["k"][1, 0, 1, 3] = 1.0
    t["q"][1] = t["k"][1]
    state = t["state"].clone()
    o = _step(t, state, o_dtype=F32)
    assert torch.equal(state[0, 0], t["state"][0, 0])
    g = float(np.exp(-5.0))
    assert float((state[0, 1] / t["state"][0, 1] - g).abs().max()) <= 8 * 2.0 ** -24 * g
    assert float((o[1, 0] - t["v"][1, 0].float()).abs().max()) <= 2.0 ** -22 * 6   # |v|, |S| below 6


def test_a_prompt_in_chunks_then_steps():
    B, T, H, dk, dv, steps = 2, 200, 2, 128, 128, 5
    t = _tokens(B, T + steps, H, dk, dv, seed=9)
    o, _, hT, _ = _oracle(t, bdla.BOUNDED)
    cut = lambda x, a, e: x[:, a:e].contiguous()
    pre, state = bdla.fwd_delta(*(cut(t[x], 0, T) for x in ("q", "k", "v", "a", "beta")), h0=t["state"])
    rest = _step(t, state, first=T)
    assert_close("prompt", pre.float().cpu().numpy(), o[:, :T].numpy())
    assert_close("steps", rest.float().cpu().numpy(), o[:, T:].numpy())
    assert_close("state", state.cpu().numpy(), hT.numpy())


def test_another_stream_and_a_replayed_graph():
    t = _tokens(6, 1, 3, 128, 128, seed=10)
    want = [t["state"].clone()]
    outs = []
    for _ in range(3):
        s = want[-1].clone()
        outs.append(_step(t, s))
        want.append(s)
    side, state = torch.cuda.Stream(), t["state"].clone()
    torch.cuda.synchronize()
    o = _step(t, state, stream=side)
    side.synchronize()
    assert torch.equal(o, outs[0]) and torch.equal(state, want[1])
    ws = bdla.Workspace(256, "cuda")
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    state = t["state"].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = bdla.decode_delta(t["q"], t["k"], t["v"], t["a"], t["beta"], state, slots=slots, ws=ws)
    for n in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, outs[n]) and torch.equal(state, want[n + 1]), n
    slots[2] = 17
    graph.replay()
    assert ws.read_device_status() == bdla.ERR_DEVICE


def test_a_pool_past_32_bit_offsets():
    """4200 states of 32 heads: 2.2e9 elements."""
    H, d = 32, 128
    pool = torch.empty((4200, H, d, d), device="cuda")
    t = _tokens(2, 1, H, d, d, seed=11)
    want = t["state"].clone()
    want_o = _step(t, want)
    slots = torch.tensor([4199, 4096], dtype=torch.int32, device="cuda")
    pool[slots.long()] = t["state"]
    o = _step(t, pool, slots=slots, ws=bdla.Workspace(256, "cuda"))
    assert torch.equal(o, want_o) and torch.equal(pool[slots.long()], want)


def test_arguments_are_refused_by_name():
    t = _tokens(2, 1, 2, 64, 64)
    order = ("q", "k", "v", "a", "beta", "state")
    for change in (dict(k=t["k"][:1]), dict(v=t["v"].float()), dict(a=t["a"].to(BF16)), dict(beta=t["beta"][0]),
                   dict(state=t["state"][:1]), dict(state=t["state"].double()), dict(state=t["state"].transpose(2, 3)),
                   dict(q=t["q"].cpu())):
        with pytest.raises(ValueError, match=next(iter(change))):
            bdla.decode_delta(*(change.get(x, t[x]) for x in order))
    args = [t[x] for x in order]
    with pytest.raises(ValueError, match="slots"):
        bdla.decode_delta(*args, slots=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="counts"):
        bdla.decode_delta(*args, counts=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="out"):
        bdla.decode_delta(*args, out=torch.empty((2, 1, 2, 128), dtype=BF16, device="cuda"))
    with pytest.raises(bdla.BdlaError) as e:
        bdla.decode_delta(*args, b=1.0)
    assert e.value.status == bdla.ERR_RANGE


@pytest.mark.parametrize("o_dtype", [BF16, F32])
def test_an_output_of_the_callers_is_filled(o_dtype):
    t = _tokens(5, 3, 4, 64, 128, seed=21)
    want = _step(t, t["state"].clone(), o_dtype=o_dtype)
    pool = torch.cat((t["state"], torch.zeros_like(t["state"][:2])))
    slots = torch.tensor([3, -1, 0, 1, 4], dtype=torch.int32, device="cuda")
    src = slots.long()
    buf = torch.full((7, 3, 4, 128), float("nan"), dtype=o_dtype, device="cuda")
    state = t["state"].clone()
    got = _step(t, state, out=buf[1:6])
    assert got.data_ptr() == buf[1:6].data_ptr() and torch.equal(buf[1:6], want)
    assert bool(buf[0].isnan().all()) and bool(buf[6].isnan().all())
    buf.fill_(float("nan"))
    got = _step(t, pool, slots=slots, out=buf[1:6])
    t["state"] = t["state"][src.clamp(min=0)]
    want = _step(t, t["state"], o_dtype=o_dtype)
    assert not bool(buf[2].any())   # the unused place
    for b in (0, 2, 3, 4):
        assert torch.equal(buf[1 + b], want[b]) and torch.equal(pool[src[b]], t["state"][b])
    assert bool(buf[0].isnan().all()) and bool(buf[6].isnan().all())
