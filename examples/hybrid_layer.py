"""One hybrid block pair on packed documents, trained and served.

A linear attention layer (bounded decay) and a softmax layer read the same projections of the same packed documents.
train_step() runs both forward and backward; serve() puts a prompt's keys and values into a paged cache, decodes, has a
tree of drafts verified, keeps the accepted path and decodes on.

    python examples/hybrid_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from chunked_linear_attention_bounded_gb300 import bdla  # noqa: E402

BF16 = torch.bfloat16


class Layer:
    """Weights of the two layers' norms and the workspaces of their calls."""

    def __init__(self, Hq=8, Hk=2, d=128, device="cuda"):
        self.Hq, self.Hk, self.d = Hq, Hk, d
        self.wq, self.wk = (torch.ones(d, device=device) for _ in range(2))     # softmax layer: learned
        self.unit = torch.full((d,), d ** -0.5, device=device)                  # linear layer: unit keys, scaled queries
        self.ws = {n: bdla.Workspace(256, device) for n in ("norm", "attn", "fwd", "bwd", "cache")}


def train_step(layer, qkv, a, dO, dO_linear, cu):
    """qkv [1, T, Hq + 2 Hk, d] (one projection), a [1, T, Hq] decay logits, upstream gradients of both outputs like
    [1, T, Hq, d].  Returns both outputs and the gradients of q, k, v, a and of the norms' weights."""
    Hq, Hk, ws = layer.Hq, layer.Hk, layer.ws
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:].contiguous()
    # softmax layer: norm and rotation in one pass, causal attention of every document
    qn, kn = bdla.qk_norm(q, k, layer.wq, layer.wk, cu_seqlens=cu)
    o, lse = bdla.attn_fwd(qn, kn, v, cu_seqlens=cu, ws=ws["attn"])
    dqn, dkn, dv = bdla.attn_bwd(qn, kn, v, o, lse, dO, cu_seqlens=cu, ws=ws["attn"])
    dq, dk, dwq, dwk = bdla.qk_norm_bwd(q, k, layer.wq, layer.wk, dqn, dkn, cu_seqlens=cu, ws=ws["norm"])
    # linear layer: unit keys without a rotation, its heads share the keys and values of their group
    G = Hq // Hk
    ql, kl = bdla.qk_norm(q, k, layer.unit, layer.unit, rotary=0, eps=1e-12)
    shared = lambda x: x.repeat_interleave(G, 2)
    ol, _, ck = bdla.fwd(ql, shared(kl), shared(v), a, cu_seqlens=cu, ckpt_stride=128, ckpt_dtype=BF16, ws=ws["fwd"])
    dql, dkl, dvl, da, _ = bdla.bwd(ql, shared(kl), shared(v), a, dO_linear, cu_seqlens=cu, ckpt=ck, ckpt_stride=128,
                                    ws=ws["bwd"])
    B, T, _, d = q.shape
    joined = lambda x: x.view(B, T, Hk, G, d).sum(3)
    # its gradients are fp32, and so is what the norm's gradient takes here
    dq2, dk2, _, _ = bdla.qk_norm_bwd(q, k, layer.unit, layer.unit, dql, joined(dkl), rotary=0, eps=1e-12, ws=ws["norm"])
    return o, ol, dict(q=dq + dq2, k=dk + dk2, v=dv + joined(dvl).to(BF16), a=da, wq=dwq, wk=dwk)


class Cache:
    """Pages of one layer's keys and values, handed out in order."""

    def __init__(self, sequences, tokens, Hk, d, page=16, device="cuda"):
        width = -(-tokens // page)
        self.k = torch.empty((sequences * width, page, Hk, d), dtype=BF16, device=device)
        self.v = torch.empty_like(self.k)
        self.pages = torch.randperm(sequences * width, device=device).int().view(sequences, width).contiguous()
        self.lens = torch.zeros(sequences, dtype=torch.int32, device=device)

    def append(self, k, v, ws, **chosen):
        bdla.cache_append(k, v, self.k, self.v, self.pages, self.lens, ws=ws, **chosen)

    def attend(self, q, ws, tree=None):
        return bdla.attn_cached(q, self.k, self.v, self.pages, self.lens, tree=tree, ws=ws)[0]


def serve(layer, prompt, draft, tree, depth, accepted, then):
    """prompt [1, T, Hq + 2 Hk, d]; draft [1, N, ...] with its visibility masks `tree` (int64 [1, N]) and depths
    [1, N]; `accepted`: the drafts on the verified path, in order; then [1, 1, ...]: the token that follows them.
    Returns the outputs of the prompt, the drafts and that token."""
    Hq, Hk, ws = layer.Hq, layer.Hk, layer.ws
    T, N = prompt.shape[1], draft.shape[1]
    cache = Cache(1, T + N + 8, Hk, layer.d, device=prompt.device)

    def split(x, positions=None):
        qn, kn = bdla.qk_norm(x[:, :, :Hq], x[:, :, Hq:Hq + Hk], layer.wq, layer.wk, positions=positions)
        return qn, kn, x[:, :, Hq + Hk:].contiguous()

    q, k, v = split(prompt)
    o_prompt, _ = bdla.attn_fwd(q, k, v, ws=ws["attn"])
    cache.append(k, v, ws["cache"])
    cache.lens.fill_(T)
    # the drafts: appended behind the prompt, each sees the prompt and its own path
    q, k, v = split(draft, (T + depth).int())
    cache.append(k, v, ws["cache"])
    o_draft = cache.attend(q, ws["cache"], tree)
    # the accepted path becomes consecutive
    n = len(accepted)
    rows = torch.zeros((1, N), dtype=torch.int32, device=prompt.device)
    rows[0, :n] = torch.tensor(accepted)
    cache.append(k, v, ws["cache"], rows=rows, counts=torch.full((1,), n, dtype=torch.int32, device=prompt.device))
    cache.lens.add_(n)
    q, k, v = split(then, cache.lens.view(1, 1).clone())
    cache.append(k, v, ws["cache"])
    o_then = cache.attend(q, ws["cache"])
    if ws["cache"].read_device_status() != bdla.OK:
        raise RuntimeError("a page, a length or a row was out of range")
    return o_prompt, o_draft, o_then


def main():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    layer = Layer()
    cu = torch.tensor([0, 700, 701, 2000], dtype=torch.int32, device="cuda")
    T, H = 2000, layer.Hq + 2 * layer.Hk
    o, ol, grads = train_step(layer, rn(1, T, H, layer.d).to(BF16), rn(1, T, layer.Hq),
                              rn(1, T, layer.Hq, layer.d).to(BF16), rn(1, T, layer.Hq, layer.d).to(BF16), cu)
    print("trained:", {n: tuple(x.shape) for n, x in grads.items()})
    tree = torch.tensor([[0b1, 0b11, 0b101, 0b1101, 0b10000, 0b110000]], dtype=torch.int64, device="cuda")
    depth = torch.tensor([[0, 1, 1, 2, 0, 1]], device="cuda")
    outs = serve(layer, rn(1, 500, H, layer.d).to(BF16), rn(1, 6, H, layer.d).to(BF16), tree, depth, [0, 2, 3],
                 rn(1, 1, H, layer.d).to(BF16))
    print("served:", [tuple(x.shape) for x in outs])
    assert all(bool(x.isfinite().all()) for x in (o, ol, *grads.values(), *outs))


if __name__ == "__main__":
    main()
