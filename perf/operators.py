"""Cases of the softmax-attention operators: what is timed, on which inputs, and what the outputs have to be.

A hybrid stack interleaves the library's linear attention with softmax layers over the same packed documents.  Four
operators make such a layer, for training and for serving:

  norm      per-head RMS norm of queries and keys with the position rotation in the same pass, and its gradient
  attn      causal softmax attention with grouped heads over whole (packed) documents, and its gradient
  append    new keys and values written into the pages of a cache (optionally a chosen subset of drafted rows)
  cached    attention of a sequence's newest tokens (one, or a tree of drafts) over such a cache

`run` computes an operator in plain torch operations while `own` is false and through the package while it is true;
`exact` computes it from its definition in 64 bits.
"""
import math
import random

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of one sequence far into its context: launch latency
        dict(name="norm 1 token", op="norm", B=1, T=1, docs=0, Hq=32, Hk=8, d=128, rot=128, inter=False, far=900000,
             bwd=False),
        # the 64K stage's packed documents, queries and keys read out of one fused projection
        dict(name="norm 64K packed", op="norm", B=1, T=65536, docs=8, Hq=32, Hk=8, d=128, rot=128, inter=False, far=0,
             bwd=False),
        # gradient at an odd token count, half of each 64-wide head rotated, pairs interleaved
        dict(name="norm backward 20011", op="norm", B=1, T=20011, docs=5, Hq=16, Hk=16, d=64, rot=32, inter=True,
             far=0, bwd=True),
        # three short documents, two heads: launch latency of the forward
        dict(name="attn 300 tokens", op="attn", B=1, T=300, docs=3, Hq=2, Hk=2, d=64, bwd=False),
        # the 64K stage: eight ragged documents, 32 query heads on 8 key heads
        dict(name="attn 64K packed", op="attn", B=1, T=65536, docs=8, Hq=32, Hk=8, d=128, bwd=False),
        # short odd documents, three query heads to a key head
        dict(name="attn backward 1537", op="attn", B=1, T=1537, docs=4, Hq=6, Hk=2, d=64, bwd=True),
        # the 8K stage's batch, gradient
        dict(name="attn backward 4x8K", op="attn", B=4, T=8192, docs=0, Hq=16, Hk=4, d=128, bwd=True),
        # one token of every one of 256 sequences into their pages
        dict(name="append 256x1", op="append", B=256, N=1, page=16, lo=1, hi=4096, Hk=8, d=128, pick=False),
        # accepted drafts of a few sequences, and a prompt's worth of rows
        dict(name="append 5x4093", op="append", B=5, N=4093, page=48, lo=0, hi=700, Hk=8, d=128, pick=True),
        # single-token decoding, many ragged sequences, small pages
        dict(name="cached 256x1", op="cached", B=256, N=1, page=16, lo=1, hi=8192, Hq=32, Hk=8, d=128, tree=False),
        # single-token decoding of one sequence over the 256K stage's context: few rows, a long axis
        dict(name="cached 1x1 256K", op="cached", B=1, N=1, page=64, lo=262143, hi=262143, Hq=32, Hk=8, d=128,
             tree=False),
        # a drafted tree verified over medium contexts, one of them empty
        dict(name="cached tree 4x61", op="cached", B=4, N=61, page=32, lo=0, hi=16384, Hq=16, Hk=4, d=128, tree=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "attn", "attn", "append", "cached", "cached"])
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 8])
    if op == "norm":
        T = _log(rng, 1, 65536 if Hk * (G + 1) <= 40 else 20000)
        docs = rng.choice([0, min(T, rng.randint(1, 9))])
        return dict(op=op, B=1 if docs else rng.choice([1, 1, 2]), T=T, docs=docs, Hq=Hk * G, Hk=Hk, d=d,
                    rot=rng.choice([0, 16, 32, 48, d // 2, d, d]), inter=rng.random() < 0.4,
                    far=0 if docs else rng.choice([0, 100000, 1 << 20]), bwd=rng.random() < 0.5)
    if op == "attn":
        bwd = rng.random() < 0.5
        T = _log(rng, 1, 16384)
        docs = rng.choice([0, min(T, rng.randint(1, 9))])
        return dict(op=op, B=1 if docs else rng.choice([1, 2, 3]), T=T, docs=docs, Hq=Hk * G, Hk=Hk, d=d, bwd=bwd)
    page = rng.choice([1, 8, 16, 24, 32, 64, 100, 128, 256])
    B = _log(rng, 1, 256)
    if op == "append":
        N = _log(rng, 1, max(1, 20000 // B))
        return dict(op=op, B=B, N=N, page=page, lo=0, hi=_log(rng, 16, 1024), Hk=Hk, d=d, pick=rng.random() < 0.5)
    hi = _log(rng, 16, max(16, min(262144, 1000000 // B)))
    tree = rng.random() < 0.5
    return dict(op=op, B=B, N=rng.randint(2, 64) if tree else rng.choice([1, 1, 1, 4]), page=page,
                lo=rng.choice([0, hi // 2]), hi=hi, Hq=Hk * G, Hk=Hk, d=d, tree=tree)


def lengths(c):
    """Tokens of each document: fixed rows, or ragged lengths that depend on the case alone."""
    if not c["docs"]:
        return [c["T"]] * c["B"]
    r = random.Random(c["T"] * 131 + c["docs"])
    n, T = c["docs"], c["T"]
    u = [r.uniform(1, 16) for _ in range(n)]
    got = [max(1, int(T * x / sum(u))) for x in u]
    got[got.index(max(got))] += T - sum(got)
    return got


def contexts(c):
    """Committed tokens of each sequence of a cache, which depend on the case alone."""
    r = random.Random(c["B"] * 977 + c["hi"])
    got = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    if c["B"] > 1:
        got[0], got[-1] = c["lo"], c["hi"]
    return got


def counts_of(c):
    """Rows that an append writes for each sequence: all of them, or between none and all."""
    r = random.Random(c["B"] * 31 + c["N"])
    got = [r.randint(0, c["N"]) if c["pick"] else c["N"] for _ in range(c["B"])]
    got[-1] = c["N"]
    return got


# ------------------------------------------------------------------ inputs
def _cache(c, g, dev, room):
    """Pages of a cache in a shuffled order, table entries past a sequence's need -1, slots never written NaN."""
    page, Hk, d = c["page"], c["Hk"], c["d"]
    lens = contexts(c)
    need = [-(-(n + room) // page) for n in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device=dev)
    width = max(need)
    at, used = torch.zeros(c["B"], dtype=torch.int64), 0
    for i, n in enumerate(need):
        at[i] = used
        used += n
    at, need = at.to(dev), torch.tensor(need, device=dev)
    j = torch.arange(width, device=dev)
    have = j[None] < need[:, None]
    table = torch.where(have, order[(at[:, None] + j[None]).clamp_max(total - 1)], -1).to(torch.int32)
    k = torch.randn((total, page, Hk, d), generator=g, device=dev, dtype=BF16)
    v = torch.randn((total, page, Hk, d), generator=g, device=dev, dtype=BF16)
    lens = torch.tensor(lens, dtype=torch.int32, device=dev)
    # slots past each sequence's end hold whatever was there
    slot = torch.arange(width * page, device=dev)[None]
    stale = (slot >= lens[:, None] + (room if c["op"] == "cached" else 0)) & have.repeat_interleave(page, 1)
    b, s = stale.nonzero(as_tuple=True)
    if b.numel():
        p = table[b, s // page].long()
        k[p, s % page] = float("nan")
        v[p, s % page] = float("nan")
    return k, v, table, lens


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 13)
    s = {"case": c}
    rn = lambda *shape: torch.randn(shape, generator=g, device=dev, dtype=BF16)
    if c["op"] in ("norm", "attn"):
        B, T, Hq, Hk, d = c["B"], c["T"], c["Hq"], c["Hk"], c["d"]
        s["lens"] = lengths(c)
        s["cu"] = None
        if c["docs"]:
            cu = [0]
            for n in s["lens"]:
                cu.append(cu[-1] + n)
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    if c["op"] == "norm":
        qkv = rn(B, T, Hq + 2 * Hk, d) * 3
        s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        s["wq"] = 1 + 0.2 * torch.randn(d, generator=g, device=dev)
        s["wk"] = 1 + 0.2 * torch.randn(d, generator=g, device=dev)
        s["pos"] = None
        if c["far"]:
            s["pos"] = torch.randint(c["far"] // 2, c["far"], (B, T), generator=g, device=dev, dtype=torch.int32)
        if c["bwd"]:
            s["dqn"], s["dkn"] = rn(B, T, Hq, d), rn(B, T, Hk, d)
        return s
    if c["op"] == "attn":
        s["q"], s["k"], s["v"] = rn(B, T, Hq, d) * 2, rn(B, T, Hk, d), rn(B, T, Hk, d)
        if c["bwd"]:
            # what the forward keeps for its gradient: its output and the log of each row's sum
            o, s["lse"] = _attn_plain(s, s["q"], s["k"], s["v"], F32)
            s["o"], s["dO"] = o.to(BF16), rn(B, T, Hq, d)
        return s
    B, N, Hk, d = c["B"], c["N"], c["Hk"], c["d"]
    s["kc"], s["vc"], s["table"], s["lens_dev"] = _cache(c, g, dev, N)
    if c["op"] == "append":
        s["k"], s["v"], s["rows"], s["counts"] = rn(B, N, Hk, d), rn(B, N, Hk, d), None, None
        if c["pick"]:
            s["counts"] = torch.tensor(counts_of(c), dtype=torch.int32, device=dev)
            # an increasing choice of drafted rows for each sequence, in its first `counts` entries
            key = torch.rand((B, N), generator=g, device=dev)
            key = torch.where(torch.arange(N, device=dev)[None] < s["counts"][:, None], key.argsort(1), N)
            s["rows"] = key.sort(1).values.clamp_max(N - 1).to(torch.int32)
        return s
    s["q"] = rn(B, N, c["Hq"], d) * 2
    s["tree"] = None
    if c["tree"]:
        # draft i's parent is an earlier draft or the context; a draft sees its ancestors and itself
        par = (torch.rand((B, N), generator=g, device=dev) * (torch.arange(N, device=dev) + 1)).long() - 1
        par = torch.minimum(par, torch.arange(N, device=dev) - 1).cpu()
        bits = torch.zeros((B, N), dtype=torch.int64)
        for i in range(N):
            mine = torch.where(par[:, i] >= 0, bits.gather(1, par[:, i].clamp_min(0)[:, None])[:, 0], 0)
            bits[:, i] = mine | ((1 << i) if i < 63 else -(1 << 63))
        if N > 4:
            bits[:, N // 2] = 0   # a padded draft: it sees the context alone, and nothing where that is empty
        s["tree"] = bits.to(dev)
    return s


# ------------------------------------------------------------------ plain forms
def _positions(s):
    c, q = s["case"], s["q"]
    if s["pos"] is not None:
        return s["pos"].double()
    t = torch.arange(c["T"], device=q.device)
    if s["cu"] is None:
        return t.double()[None].expand(c["B"], -1)
    doc = torch.bucketize(t, s["cu"][1:-1].long(), right=True)
    return (t - s["cu"].long()[doc]).double()[None]


EPS, BASE = 1e-6, 10000.0


def _angles(s):
    rot = s["case"]["rot"]
    f = BASE ** (-torch.arange(0, rot, 2, device=s["q"].device, dtype=F64) / rot)
    a = _positions(s)[..., None, None] * f
    return a.cos().float(), a.sin().float()


def _split(x, rot, inter):
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])


def _join(a, b, rest, inter):
    ab = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((ab, rest), -1)


def _norm_plain(x, w, cos, sin, rot, inter):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    if not rot:
        return y
    a, b = _split(y, rot, inter)
    return _join(a * cos - b * sin, b * cos + a * sin, y[..., rot:], inter)


def _norm_back_plain(x, w, dy, cos, sin, rot, inter):
    x, dy = x.float(), dy.float()
    if rot:
        a, b = _split(dy, rot, inter)
        dy = _join(a * cos + b * sin, b * cos - a * sin, dy[..., rot:], inter)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    h = dy * w
    dx = r * (h - n * (h * n).mean(-1, keepdim=True))
    return dx, (dy * n).sum((0, 1, 2))


def _spans(s):
    """(first token, length) of each document in the flattened tokens."""
    at, got = 0, []
    for n in s["lens"]:
        got.append((at, n))
        at += n
    return got


def _scores(q, k, scale):
    """Masked scores [G, n, n] of one document and key head, in the type of q."""
    n = q.shape[1]
    x = (q @ k.T) * scale
    i = torch.arange(n, device=q.device)
    return x.masked_fill(i[None, :] > i[:, None], float("-inf"))


def _attn_plain(s, q, k, v, kind):
    B, T, Hq, d = q.shape
    Hk = k.shape[2]
    G = Hq // Hk
    q, k, v = (x.reshape(B * T, -1, G if x is q else 1, d) for x in (q, k, v))
    o = torch.empty((B * T, Hk, G, d), dtype=kind, device=q.device)
    lse = torch.empty((Hk, G, B * T), dtype=kind, device=q.device)
    for at, n in _spans(s):
        for h in range(Hk):
            x = _scores(q[at:at + n, h].to(kind).transpose(0, 1), k[at:at + n, h, 0].to(kind), d ** -0.5)
            m = x.amax(-1, keepdim=True)
            p = (x - m).exp_()
            del x
            z = p.sum(-1, keepdim=True)
            o[at:at + n, h] = ((p @ v[at:at + n, h, 0].to(kind)) / z).transpose(0, 1)
            lse[h, :, at:at + n] = (m + z.log())[..., 0]
    return o.reshape(B, T, Hq, d), lse.reshape(Hq, B * T)


def _attn_back_plain(s, kind):
    q, k, v, dO = s["q"], s["k"], s["v"], s["dO"]
    B, T, Hq, d = q.shape
    Hk = k.shape[2]
    G = Hq // Hk
    gq = torch.empty((B * T, Hk, G, d), dtype=kind, device=q.device)
    gk = torch.empty((B * T, Hk, d), dtype=kind, device=q.device)
    gv = torch.empty((B * T, Hk, d), dtype=kind, device=q.device)
    q, dO = (x.reshape(B * T, Hk, G, d) for x in (q, dO))
    k, v = (x.reshape(B * T, Hk, d) for x in (k, v))
    for at, n in _spans(s):
        for h in range(Hk):
            qh, gh = (x[at:at + n, h].to(kind).transpose(0, 1) for x in (q, dO))
            kh, vh = k[at:at + n, h].to(kind), v[at:at + n, h].to(kind)
            x = _scores(qh, kh, d ** -0.5)
            p = (x - x.amax(-1, keepdim=True)).exp_()
            del x
            p /= p.sum(-1, keepdim=True)
            dp = gh @ vh.T
            # the row's own sum of P o dP
            dp -= (p * dp).sum(-1, keepdim=True)
            gv[at:at + n, h] = torch.einsum("gij,gid->jd", p, gh)
            dp *= p
            del p
            dp *= d ** -0.5
            gq[at:at + n, h] = (dp @ kh).transpose(0, 1)
            gk[at:at + n, h] = torch.einsum("gij,gid->jd", dp, qh)
            del dp
    return gq.reshape(B, T, Hq, d), gk.reshape(B, T, Hk, d), gv.reshape(B, T, Hk, d)


def _append_plain(s):
    c, table, lens = s["case"], s["table"], s["lens_dev"].long()
    N, page = c["N"], c["page"]
    j = torch.arange(N, device=lens.device)
    at = lens[:, None] + j[None]
    slot = table.long().gather(1, at // page) * page + at % page
    k, v = s["k"], s["v"]
    if s["rows"] is not None:
        pick = s["rows"].long()[..., None, None].expand_as(k)
        k, v = k.gather(1, pick), v.gather(1, pick)
        live = (j[None] < s["counts"][:, None])[..., None, None]
        flat = slot.reshape(-1)
        k = torch.where(live, k, s["kc"].flatten(0, 1)[flat].view_as(k))
        v = torch.where(live, v, s["vc"].flatten(0, 1)[flat].view_as(v))
    s["kc"].view(-1, *k.shape[2:]).index_copy_(0, slot.reshape(-1), k.flatten(0, 1))
    s["vc"].view(-1, *v.shape[2:]).index_copy_(0, slot.reshape(-1), v.flatten(0, 1))
    return s["kc"], s["vc"]


def _cached_group(s, b0, b1, kind):
    """Sequences b0 .. b1 - 1: outputs [b, N, Hq, d] and log-sums [b, N, Hq]."""
    c, dev = s["case"], s["q"].device
    N, Hk, d, page = c["N"], c["Hk"], c["d"], c["page"]
    G, n = c["Hq"] // Hk, b1 - b0
    lens = s["lens_dev"][b0:b1].long()
    slot = torch.arange(s["table"].shape[1] * page, device=dev)
    have = slot[None] < lens[:, None] + N
    pages = s["table"][b0:b1].long().clamp_min(0)
    gather = lambda x: x[pages].flatten(1, 2).to(kind).masked_fill(~have[..., None, None], 0)   # [n, S, Hk, d]
    k, v = gather(s["kc"]), gather(s["vc"])
    i, draft = torch.arange(N, device=dev), slot[None] - lens[:, None]
    if s["tree"] is None:
        see = draft[:, None] <= i[None, :, None]
    else:
        bit = (s["tree"][b0:b1][:, :, None] >> draft.clamp(0, 63)[:, None]) & 1
        see = (draft[:, None] < 0) | ((bit == 1) & (draft[:, None] < N))
    see = (see & have[:, None])[:, None, None]                                                   # [n, 1, 1, N, S]
    q = s["q"][b0:b1].reshape(n, N, Hk, G, d).to(kind)
    x = torch.einsum("bnhgd,bshd->bhgns", q, k) * d ** -0.5
    x = x.masked_fill(~see, float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = (x - m.clamp_min(torch.finfo(kind).min)).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgns,bshd->bnhgd", p / torch.where(z > 0, z, 1), v)
    lse = (m + z.log())[..., 0].permute(0, 3, 1, 2)
    return o.reshape(n, N, -1, d), lse.reshape(n, N, -1)


def _cached_plain(s, kind):
    c = s["case"]
    cap = s["table"].shape[1] * c["page"]
    step = max(1, (1 << 31) // (cap * max(c["Hk"] * c["d"], c["Hq"] * c["N"])))
    parts = [_cached_group(s, b, min(c["B"], b + step), kind) for b in range(0, c["B"], step)]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "norm":
        cos, sin = _angles(s)
        if not c["bwd"]:
            return tuple(_norm_plain(s[x], s["w" + x], cos, sin, c["rot"], c["inter"]).to(BF16) for x in "qk")
        (dq, dwq), (dk, dwk) = (_norm_back_plain(s[x], s["w" + x], s["d%sn" % x], cos, sin, c["rot"], c["inter"])
                                for x in "qk")
        return dq.to(BF16), dk.to(BF16), dwq, dwk
    if c["op"] == "attn":
        if c["bwd"]:
            return tuple(x.to(BF16) for x in _attn_back_plain(s, F32))
        o, lse = _attn_plain(s, s["q"], s["k"], s["v"], F32)
        return o.to(BF16), lse
    if c["op"] == "append":
        return _append_plain(s)
    o, lse = _cached_plain(s, F32)
    return o.to(BF16), lse


def _run_own(s, c):
    from chunked_linear_attention_bounded_gb300 import bdla
    if "ws" not in s:
        s["ws"] = bdla.Workspace(256, s["q" if "q" in s else "k"].device)   # kept from call to call, as a program does
    ws = s["ws"]
    if c["op"] == "norm":
        kw = dict(rotary=c["rot"], base=BASE, interleaved=c["inter"], positions=s["pos"], cu_seqlens=s["cu"], eps=EPS)
        if not c["bwd"]:
            return bdla.qk_norm(s["q"], s["k"], s["wq"], s["wk"], **kw)
        return bdla.qk_norm_bwd(s["q"], s["k"], s["wq"], s["wk"], s["dqn"], s["dkn"], ws=ws, **kw)
    if c["op"] == "attn":
        if c["bwd"]:
            return bdla.attn_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dO"], cu_seqlens=s["cu"], ws=ws)
        return bdla.attn_fwd(s["q"], s["k"], s["v"], cu_seqlens=s["cu"], ws=ws)
    if c["op"] == "append":
        bdla.cache_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens_dev"], rows=s["rows"],
                          counts=s["counts"], ws=ws)
        return s["kc"], s["vc"]
    return bdla.attn_cached(s["q"], s["kc"], s["vc"], s["table"], s["lens_dev"], tree=s["tree"], ws=ws)


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "append":
        return None
    if c["op"] == "norm":
        return _norm_exact(c, s)
    if c["op"] == "attn":
        pairs = sum(n * n for n in lengths(c)) * c["Hq"] * c["d"]
        if pairs * (10 if c["bwd"] else 4) > 1.5e13:
            return None
        return _attn_exact(c, s)
    return _cached_exact(c, s)


def _turn(c, s):
    """The rotation as one complex factor for each token and pair."""
    B, T, dev = c["B"], c["T"], s["q"].device
    if s["pos"] is not None:
        pos = s["pos"].double()
    else:
        pos = torch.cat([torch.arange(n, dtype=F64, device=dev) for n in s["lens"]]).view(B, T)
    i = torch.arange(c["rot"] // 2, dtype=F64, device=dev)
    ang = pos[..., None] / BASE ** (2 * i / c["rot"])
    return torch.polar(torch.ones_like(ang), ang)[:, :, None]


def _as_complex(y, c):
    r = y[..., :c["rot"]]
    r = r.reshape(*r.shape[:-1], -1, 2) if c["inter"] else r.reshape(*r.shape[:-1], 2, -1).transpose(-1, -2)
    return torch.view_as_complex(r.contiguous())


def _from_complex(z, c):
    r = torch.view_as_real(z)
    return (r if c["inter"] else r.transpose(-1, -2)).flatten(-2)


def _norm_exact(c, s):
    turn = _turn(c, s) if c["rot"] else None
    outs, grads = [], []
    for x in "qk":
        u, w = s[x].double(), s["w" + x].double()
        length = ((u ** 2).sum(-1, keepdim=True) / c["d"] + EPS) ** 0.5
        if not c["bwd"]:
            y = u / length * w
            if c["rot"]:
                y[..., :c["rot"]] = _from_complex(_as_complex(y, c) * turn, c)
            outs.append(y)
            continue
        dy = s["d%sn" % x].double()
        if c["rot"]:
            dy[..., :c["rot"]] = _from_complex(_as_complex(dy, c) * turn.conj(), c)
        # y_i = w_i u_i / length, so dL/du_j = w_j dy_j / length - u_j (sum_i w_i dy_i u_i) / (d length^3)
        outs.append(dy * w / length - u * (dy * w * u).sum(-1, keepdim=True) / (c["d"] * length ** 3))
        grads.append((dy * u / length).sum((0, 1, 2)))
    return tuple(outs + grads)


def _attn_exact(c, s):
    """Row blocks against the keys up to their end, each score from the definition."""
    B, T, Hq, Hk, d = c["B"], c["T"], c["Hq"], c["Hk"], c["d"]
    G, dev = Hq // Hk, s["q"].device
    flat = lambda x: x.reshape(B * T, -1, d)
    q, k, v = flat(s["q"]), flat(s["k"]), flat(s["v"])
    outs = {x: torch.zeros((B * T, h, d), dtype=F64, device=dev) for x, h in (("o", Hq), ("dq", Hq), ("dk", Hk), ("dv", Hk))}
    lse = torch.zeros((Hq, B * T), dtype=F64, device=dev)
    at = 0
    for n in lengths(c):
        for h in range(Hq):
            kk, vv = k[at:at + n, h // G].double(), v[at:at + n, h // G].double()
            for r0 in range(0, n, 2048):
                r1 = min(n, r0 + 2048)
                qq = q[at + r0:at + r1, h].double()
                w = torch.tril(torch.ones((r1 - r0, r1), dtype=torch.bool, device=dev), diagonal=r0)
                x = qq @ kk[:r1].T / math.sqrt(d)
                l = torch.logsumexp(torch.where(w, x, -math.inf), 1)
                lse[h, at + r0:at + r1] = l
                p = torch.where(w, torch.exp(x - l[:, None]), 0.0)
                del x
                o = p @ vv[:r1]
                outs["o"][at + r0:at + r1, h] = o
                if c["bwd"]:
                    g = flat(s["dO"])[at + r0:at + r1, h].double()
                    outs["dv"][at:at + r1, h // G] += p.T @ g
                    ds = p * (g @ vv[:r1].T - (g * o).sum(1, keepdim=True)) / math.sqrt(d)
                    outs["dq"][at + r0:at + r1, h] = ds @ kk[:r1]
                    outs["dk"][at:at + r1, h // G] += ds.T @ qq
        at += n
    if c["bwd"]:
        return tuple(outs[x].view(B, T, -1, d) for x in ("dq", "dk", "dv"))
    return outs["o"].view(B, T, Hq, d), lse


def _cached_exact(c, s):
    N, Hq, Hk, d, page = c["N"], c["Hq"], c["Hk"], c["d"], c["page"]
    dev = s["q"].device
    o = torch.zeros((c["B"], N, Hq, d), dtype=F64, device=dev)
    lse = torch.full((c["B"], N, Hq), -math.inf, dtype=F64, device=dev)
    table = s["table"].cpu()
    tree = s["tree"].cpu() if s["tree"] is not None else None
    for b, n in enumerate(contexts(c)):
        used = table[b, :-(-(n + N) // page)].long().to(dev)
        k = s["kc"][used].flatten(0, 1)[:n + N].double()
        v = s["vc"][used].flatten(0, 1)[:n + N].double()
        see = torch.ones((N, n + N), dtype=torch.bool)
        for i in range(N):
            for j in range(N):
                see[i, n + j] = j <= i if tree is None else bool((int(tree[b, i]) >> j) & 1)
        see, some = see.to(dev), see.any(1).to(dev)
        for h in range(Hk):
            a, e = h * (Hq // Hk), (h + 1) * (Hq // Hk)
            x = torch.einsum("ngd,sd->ngs", s["q"][b, :, a:e].double(), k[:, h]) / math.sqrt(d)
            x = torch.where(see[:, None], x, -math.inf)
            l = torch.logsumexp(x, -1)
            p = torch.where(some[:, None, None], torch.exp(x - torch.where(some[:, None], l, 0.0)[..., None]), 0.0)
            o[b, :, a:e] = torch.einsum("ngs,sd->ngd", p, v[:, h])
            lse[b, :, a:e] = l
    return o, lse


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "norm":
        el = c["B"] * c["T"] * (c["Hq"] + c["Hk"]) * c["d"]
        # forward: read x, write y; backward: read x and dy, write dx
        return {"bytes": el * 2 * (3 if c["bwd"] else 2), "flops": el * (14 if c["bwd"] else 7)}
    if c["op"] == "attn":
        tok, d = c["B"] * c["T"], c["d"]
        pairs = sum(n * (n + 1) // 2 for n in lengths(c)) * c["Hq"]
        qb, kb = tok * c["Hq"] * d * 2, tok * c["Hk"] * d * 2
        if c["bwd"]:   # five products of the pairs; q, o, dO, dq and k, v, dk, dv once, the log-sums
            return {"bytes": 4 * qb + 4 * kb + tok * c["Hq"] * 4, "flops": pairs * d * 10}
        return {"bytes": 2 * qb + 2 * kb + tok * c["Hq"] * 4, "flops": pairs * d * 4}
    row = c["Hk"] * c["d"] * 2
    if c["op"] == "append":
        return {"bytes": sum(counts_of(c)) * row * 4, "flops": 0}
    keys = sum(contexts(c)) + c["B"] * c["N"]
    qb = c["B"] * c["N"] * c["Hq"] * c["d"] * 2
    return {"bytes": keys * row * 2 + 2 * qb, "flops": keys * c["N"] * c["Hq"] * c["d"] * 4}
