"""The serving example: a prompt once, then steps, verified drafts and steps again, each output against the definition over
the sample's whole sequence."""
import os
import sys

import numpy as np
import pytest
import torch

import _attn_ref as ref
import oracle

from _parity import assert_close

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import sample_batch  # noqa: E402

pytestmark = pytest.mark.gpu


def test_the_example_runs():
    sample_batch.main()


@pytest.mark.parametrize("T", [203, 32, 5])   # past whole pages, whole pages alone, less than a page
def test_samples_are_what_their_whole_sequences_give(T):
    n, d, Hq, Hk, H = 6, 128, 8, 2, 4
    s = sample_batch.Samples(n, T, room=40)
    prompt = sample_batch.inputs(1, T, seed=20)
    steps = [sample_batch.inputs(n, 1, seed=21 + i) for i in range(2)]
    drafts, last = sample_batch.inputs(n, 4, seed=30), sample_batch.inputs(n, 1, seed=31)
    kept = torch.tensor([0, 4, 2, 1, 3, 4], dtype=torch.int32, device="cuda")
    o, od = s.prefill(*prompt)
    got = [s.step(*x) for x in steps]
    got_drafts = s.step(*drafts, keep=0)
    before = s.states.clone()
    s.settle(kept, *drafts[1:])
    got_last = s.step(*last)
    s.check()
    assert not torch.equal(before, s.states) and s.lens.tolist() == [T + 3 + int(x) for x in kept]
    for b in range(n):
        # everything that the sample has seen: all drafts for the drafts' outputs, the kept ones for the last step's
        def whole(i, m, tail):
            parts = [prompt[i][0]] + [x[i][b] for x in steps] + [drafts[i][b][:m]] + ([last[i][b]] if tail else [])
            return torch.cat(parts)[None]

        for m, tail, softmax, delta, at, count in ((4, False, got_drafts[0][b], got_drafts[1][b], T + 2, 4),
                                                   (int(kept[b]), True, got_last[0][b], got_last[1][b], T + 2 + int(kept[b]), 1)):
            qkv = whole(0, m, tail)
            L = qkv.shape[1]
            R = ref.rotation(ref.positions(1, L, None, "cuda"), d, 10000.0, d, False)
            (qn, _), (kn, _) = (ref.norm(x, torch.ones(d, device="cuda"), R, 1e-6) for x in (qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]))
            want = ref.attn(qn, kn, qkv[:, :, Hq + Hk:].double(), d ** -0.5)["o"][0][0]
            # q and k are rounded to bf16 on the way: half a step of each in every score, a few of them in an output
            assert_close("softmax", softmax.float().cpu().numpy(), want[at:at + count].cpu().numpy(), rel=2e-2, max_abs=5e-2)
            if m == 4 and b == 0:
                assert_close("prompt", o[0].float().cpu().numpy(), want[:T].cpu().numpy(), rel=2e-2, max_abs=5e-2)
                assert_close("step", torch.stack([g[0][b, 0] for g in got]).float().cpu().numpy(), want[T:T + 2].cpu().numpy(),
                             rel=2e-2, max_abs=5e-2)
            f = lambda i: whole(i, m, tail)[0].double().cpu().numpy()
            want_d, _ = oracle.fwd_delta(f(1), f(2), f(3), f(4), f(5), -5.0, 0, cu_seqlens=np.array([0, L]))
            assert_close("delta", delta.float().cpu().numpy(), want_d[at:at + count])


@pytest.mark.parametrize("T", [203, 32])
def test_samples_whose_prompt_is_read_once(T):
    """At these sizes a call joins nothing by itself."""
    sample_batch.bdla.set_share_least(0)
    try:
        test_samples_are_what_their_whole_sequences_give(T)
    finally:
        sample_batch.bdla.set_share_least(-1)


@pytest.mark.parametrize("n,T,least,once", [(12, 403, -1, True), (6, 203, -1, False), (6, 203, 0, True)])
def test_whether_a_step_reads_the_prompt_once(n, T, least, once):
    """What is read once is read as the first sample's table says: without the others' entries the outputs are the same.
    The first size is the example's own."""
    outs = []
    for cut in (False, True):
        s = sample_batch.Samples(n, T, room=40)
        s.prefill(*sample_batch.inputs(1, T, seed=41))
        if cut:
            s.pages[1:, :s.whole] = -1
        sample_batch.bdla.set_share_least(least)
        try:
            outs.append(s.step(*sample_batch.inputs(n, 1, seed=42)))
        finally:
            sample_batch.bdla.set_share_least(-1)
        assert s.ws.read_device_status() == (sample_batch.bdla.ERR_DEVICE if cut and not once else sample_batch.bdla.OK)
    assert torch.equal(outs[0][1], outs[1][1]) and torch.equal(outs[0][0][:1], outs[1][0][:1])
    assert torch.equal(outs[0][0], outs[1][0]) == once
