"""Several continuations of one prompt, served from resident states and a shared cache.

A delta-rule layer and a softmax layer of a hybrid stack.  The prompt runs once, whole.  Its state is copied to a slot for
each sample, and the samples' page tables begin with the prompt's pages; a page that the prompt leaves part empty is copied.
Then every step is three calls: queries and keys normed, rotated and appended; attention that reads the prompt's whole pages
once for all samples (where that saves enough, as here: bdla.set_share_least); a recurrent step of the delta rule.  A drafted chain is verified by the same calls over several tokens: the states
stay where they are until it is known how many drafts are kept.

    python examples/sample_batch.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from chunked_linear_attention_bounded_gb300 import bdla  # noqa: E402

BF16 = torch.bfloat16


class Samples:
    """`n` samples of up to `room` tokens behind a prompt, for one layer of each kind."""

    def __init__(self, n, prompt_tokens, room, Hq=8, Hk=2, H=4, d=128, page=16, device="cuda"):
        self.n, self.Hq, self.Hk, self.page = n, Hq, Hk, page
        self.wq, self.wk = (torch.ones(d, device=device) for _ in range(2))
        self.ws = bdla.Workspace(256, device)
        # pages: the prompt's, which all samples share as far as they are full, then each sample's own
        self.whole = prompt_tokens // page
        own = -(-(prompt_tokens + room) // page) - self.whole
        self.k = torch.empty((self.whole + 1 + n * own, page, Hk, d), dtype=BF16, device=device)
        self.v = torch.empty_like(self.k)
        i32 = dict(dtype=torch.int32, device=device)
        self.prompt_pages = torch.arange(self.whole + 1, **i32)[None]
        mine = self.whole + 1 + torch.arange(n * own, **i32).view(n, own)
        self.pages = torch.cat((self.prompt_pages[:, :self.whole].expand(n, -1), mine), 1).contiguous()
        self.lens = torch.zeros(n, **i32)
        self.groups, self.shared = torch.tensor([0, n], **i32), torch.tensor([self.whole * page], **i32)
        self.states = torch.zeros((n, H, d, d), device=device)
        self.slots = torch.randperm(n, device=device).int()   # samples may live anywhere in the pool

    def prefill(self, qkv, q, k, v, a, beta):
        """The prompt: qkv [1, T, Hq + 2 Hk, d] of the softmax layer; q, k, v [1, T, H, d], a, beta [1, T, H] of the other.
        Returns both layers' outputs."""
        Hq, Hk, T = self.Hq, self.Hk, qkv.shape[1]
        qn, kn = bdla.qk_norm(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], self.wq, self.wk)
        values = qkv[:, :, Hq + Hk:].contiguous()
        o, _ = bdla.attn_fwd(qn, kn, values, ws=self.ws)
        empty = torch.zeros(1, dtype=torch.int32, device=qkv.device)
        bdla.cache_append(kn, values, self.k, self.v, self.prompt_pages, empty, ws=self.ws)
        first = self.pages[:, self.whole].long()   # a page that is not full goes to every sample
        for cache in (self.k, self.v):
            cache[first] = cache[self.whole].clone()
        self.lens.fill_(T)
        od, state = bdla.fwd_delta(q, k, v, a, beta, ws=self.ws)
        self.states.copy_(state.expand_as(self.states))
        return o, od

    def step(self, qkv, q, k, v, a, beta, keep=None):
        """T new tokens of every sample ([n, T, ...] each).  Without `keep` they are all kept.  With keep = 0 they are
        drafts, and the call leaves everything as it was; settle() keeps some of them."""
        Hq, Hk = self.Hq, self.Hk
        qn = bdla.qk_norm_append(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:], self.wq, self.wk, self.k, self.v,
                                 self.pages, self.lens, ws=self.ws)
        o, _ = bdla.attn_shared(qn, self.k, self.v, self.pages, self.lens, self.groups, self.shared, ws=self.ws)
        counts = None if keep is None else torch.zeros_like(self.lens)
        od = bdla.decode_delta(q, k, v, a, beta, self.states, slots=self.slots, counts=counts, ws=self.ws)
        if keep is None:
            self.lens.add_(qkv.shape[1])
        return o, od

    def settle(self, kept, q, k, v, a, beta):
        """Keeps the first kept[b] (int32 [n]) of the drafts that step() has seen: their keys and values are in place, and
        the states take them in."""
        bdla.decode_delta(q, k, v, a, beta, self.states, slots=self.slots, counts=kept, ws=self.ws)
        self.lens.add_(kept)

    def check(self):
        if self.ws.read_device_status() != bdla.OK:
            raise RuntimeError("a page, a length or a slot was out of range")


def inputs(n, T, Hq=8, Hk=2, H=4, d=128, seed=1, device="cuda"):
    """Random projections of T tokens of n sequences: (qkv, q, k, v, a, beta)."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=device)
    k = rn(n, T, H, d)
    return (rn(n, T, Hq + 2 * Hk, d).to(BF16), (rn(n, T, H, d) * d ** -0.5).to(BF16), (k / k.norm(dim=-1, keepdim=True)).to(BF16),
            rn(n, T, H, d).to(BF16), rn(n, T, H) - 2, torch.rand((n, T, H), generator=g, device=device))


def main():
    n, T = 12, 403
    s = Samples(n, T, room=40)
    outs = [*s.prefill(*inputs(1, T, seed=1))]
    for i in range(3):
        outs += s.step(*inputs(n, 1, seed=2 + i))
    drafts = inputs(n, 5, seed=9)
    outs += s.step(*drafts, keep=0)
    s.settle(torch.arange(n, dtype=torch.int32, device="cuda") % 6, *drafts[1:])
    outs += s.step(*inputs(n, 1, seed=10))
    s.check()
    print("served:", [tuple(x.shape) for x in outs], "tokens:", s.lens.tolist())
    assert all(bool(x.isfinite().all()) for x in outs)


if __name__ == "__main__":
    main()
