"""Cases of the operators of a serving step: what is timed, on which inputs, and what the outputs have to be.

A hybrid stack that serves holds two things for each sequence: the recurrent states of its delta-rule layers and the
paged caches of its softmax layers.  Three operators move them on by a step:

  delta    the gated delta rule from a resident state, for one new token or a few, with states in a pool
  append   queries and keys normed and rotated, keys and values written into the pages of a cache, in one call
  shared   attention of the newest tokens over such a cache, where groups of sequences share a long prefix

`run` computes an operator in plain torch operations while `own` is false and through the package while it is true;
`exact` computes it from its definition in 64 bits.
"""
import math
import random

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS, BASE, BOUND = 1e-6, 10000.0, -5.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of one sequence: launch latency
        dict(name="delta 1x1", op="delta", B=1, T=1, H=32, dk=128, dv=128, soft=False, pool=0, pad=0, count=False,
             f32=False),
        # a decode step of a large batch whose states lie anywhere in a pool, three places of the batch unused
        dict(name="delta 256x1", op="delta", B=256, T=1, H=32, dk=128, dv=128, soft=False, pool=40, pad=3, count=False,
             f32=False),
        # short drafted chains of which each sequence keeps a part, narrow keys, the unbounded decay
        dict(name="delta 37x5 kept", op="delta", B=37, T=5, H=12, dk=64, dv=128, soft=True, pool=1, pad=0, count=True,
             f32=True),
        # a prompt's short rest run through the recurrence
        dict(name="delta 48x33", op="delta", B=48, T=33, H=16, dk=128, dv=64, soft=False, pool=0, pad=0, count=False,
             f32=False),
        # a decode step of one sequence far into its context
        dict(name="append 1x1", op="append", B=1, T=1, packed=False, lo=900000, hi=900000, page=64, Hq=32, Hk=8, d=128,
             rot=128, inter=False, pick=False, queries=True),
        # a decode step of a large batch
        dict(name="append 256x1", op="append", B=256, T=1, packed=False, lo=1, hi=8192, page=16, Hq=32, Hk=8, d=128,
             rot=128, inter=False, pick=False, queries=True),
        # eight ragged prompts at the 64K stage's size, some behind a context
        dict(name="append 64K packed", op="append", B=8, T=65536, packed=True, lo=0, hi=5000, page=32, Hq=32, Hk=8,
             d=128, rot=128, inter=False, pick=False, queries=True),
        # the accepted of each sequence's drafts, pages that are no power of two, a quarter of each head rotated
        dict(name="append 91x61 picked", op="append", B=91, T=61, packed=False, lo=0, hi=700, page=48, Hq=16, Hk=16,
             d=64, rot=16, inter=True, pick=True, queries=True),
        # eight samples from one short prompt: launch latency
        dict(name="shared 8x1 2K", op="shared", B=8, T=1, groups=1, loose=0, plo=2048, phi=2048, lo=1, hi=300, page=16,
             Hq=16, Hk=4, d=128, tree=False),
        # a large batch behind one long system prompt
        dict(name="shared 256x1 32K", op="shared", B=256, T=1, groups=1, loose=0, plo=32768, phi=32768, lo=1, hi=512,
             page=64, Hq=32, Hk=8, d=128, tree=False),
        # few samples over a very long document: few rows, a long axis
        dict(name="shared 16x1 128K", op="shared", B=16, T=1, groups=1, loose=0, plo=131072, phi=131072, lo=200, hi=2000,
             page=64, Hq=32, Hk=8, d=128, tree=False),
        # trees of drafts over five prompts of unequal length and use, and three sequences of their own
        dict(name="shared tree 29x17", op="shared", B=29, T=17, groups=5, loose=3, plo=0, phi=16384, lo=0, hi=2000,
             page=48, Hq=12, Hk=4, d=64, tree=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["delta", "append", "shared"])
    if op == "delta":
        H, dk, dv = rng.choice([1, 2, 5, 8, 12, 16, 32]), rng.choice([64, 128]), rng.choice([64, 128])
        T = rng.choice([1, 1, rng.randint(2, 8), rng.randint(9, 64)])
        B = _log(rng, 1, min(256, 256 * 32 // H // max(1, T // 4)))
        pool = rng.choice([0, rng.randint(1, 9)])
        return dict(op=op, B=B, T=T, H=H, dk=dk, dv=dv, soft=rng.random() < 0.4, pool=pool,
                    pad=rng.randint(0, B // 4) if pool else 0, count=rng.random() < 0.4, f32=rng.random() < 0.3)
    Hk, G, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128])
    page = rng.choice([1, 8, 16, 24, 32, 64, 100, 128, 256])
    if op == "append":
        while Hk * (G + 2) > 48:
            G -= 1
        packed = rng.random() < 0.4
        B = _log(rng, 1, 64 if packed else 256)
        T = max(B, _log(rng, 1, 65536)) if packed else _log(rng, 1, max(1, 40000 // B))
        pick = not packed and rng.random() < 0.4
        hi = _log(rng, 16, 1 << 20 if page > 8 else 20000)
        return dict(op=op, B=B, T=T, packed=packed, lo=rng.choice([0, hi // 2]), hi=hi, page=page, Hq=Hk * G, Hk=Hk, d=d,
                    rot=rng.choice([0, 16, 32, 48, d // 2, d, d]), inter=rng.random() < 0.4, pick=pick,
                    queries=not pick or rng.random() < 0.7)
    B = _log(rng, 1, 256)
    tree = rng.random() < 0.4
    T = rng.randint(2, max(2, min(64, 600 // B))) if tree else rng.choice([1, 1, 1, 3])
    groups = rng.randint(1, min(B, 6))
    phi = _log(rng, 64, min(131072, 7000000 // (B * T)))
    hi = _log(rng, 16, min(4096, max(16, 120000 // B)))
    return dict(op=op, B=B, T=T, groups=groups, loose=rng.randint(0, B - groups) if rng.random() < 0.3 else 0,
                plo=rng.choice([0, phi // 2, phi]), phi=phi, lo=rng.choice([0, hi // 2]), hi=hi, page=page,
                Hq=Hk * G, Hk=Hk, d=d, tree=tree)


def _spread(seed, n, lo, hi):
    """n lengths in lo .. hi, both ends among them, which depend on the case alone."""
    r = random.Random(seed)
    got = [r.randint(lo, hi) for _ in range(n)]
    if n > 1:
        got[0], got[-1] = lo, hi
    return got


def contexts(c):
    """Tokens that each sequence has in the cache (behind the shared prefix, where there is one)."""
    return _spread(c["B"] * 977 + c["hi"], c["B"], c["lo"], c["hi"])


def news(c):
    """New tokens of each sequence of an append."""
    if not c["packed"]:
        return [c["T"]] * c["B"]
    r = random.Random(c["T"] * 131 + c["B"])
    u = [r.uniform(1, 16) for _ in range(c["B"])]
    got = [max(1, int((c["T"] - c["B"]) * x / sum(u))) for x in u]
    got[got.index(max(got))] += c["T"] - sum(got)
    return got


def kept(c):
    """Rows that an append writes, or tokens that a state absorbs, of each sequence: all, or between none and all."""
    if not c.get("pick") and not c.get("count"):
        return None
    return _spread(c["B"] * 31 + c["T"], c["B"], 0, c["T"])


def members(c):
    """(first sequence, sequences, prefix length) of each group; the loose sequences are the last."""
    r = random.Random(c["B"] * 53 + c["phi"])
    n, B = c["groups"], c["B"] - c["loose"]
    cuts = [0] + sorted(r.sample(range(1, B), n - 1)) + [B] if n > 1 else [0, B]
    prefix = _spread(c["phi"] * 7 + n, n, c["plo"], c["phi"])
    prefix[-1] = c["phi"]
    return [(cuts[g], cuts[g + 1] - cuts[g], prefix[g]) for g in range(n)]


# ------------------------------------------------------------------ inputs
def _trees(g, B, T, dev):
    """Visibility masks: draft i's parent is an earlier draft or the context; a draft sees its ancestors and itself."""
    par = (torch.rand((B, T), generator=g, device=dev) * (torch.arange(T, device=dev) + 1)).long() - 1
    par = torch.minimum(par, torch.arange(T, device=dev) - 1).cpu()
    bits = torch.zeros((B, T), dtype=torch.int64)
    for i in range(T):
        mine = torch.where(par[:, i] >= 0, bits.gather(1, par[:, i].clamp_min(0)[:, None])[:, 0], 0)
        bits[:, i] = mine | ((1 << i) if i < 63 else -(1 << 63))
    if T > 4:
        bits[:, T // 2] = 0   # a padded draft: it sees the context alone, and nothing where that is empty
    return bits.to(dev)


def _prepare_delta(c, g, dev, s, rn):
    B, T, H, dk, dv = (c[x] for x in ("B", "T", "H", "dk", "dv"))
    k = torch.randn((B, T, H, dk), generator=g, device=dev)
    s["q"], s["v"] = (rn(B, T, H, dk) * dk ** -0.5), rn(B, T, H, dv)
    s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(BF16)
    s["a"] = torch.randn((B, T, H), generator=g, device=dev) * 1.5 - 3
    s["beta"] = torch.rand((B, T, H), generator=g, device=dev)
    n = B + c["pool"]
    s["state"] = torch.randn((n, H, dk, dv), generator=g, device=dev) * 0.3
    s["slots"] = s["counts"] = None
    if c["pool"]:
        slots = torch.randperm(n, generator=g, device=dev)[:B].int()
        if c["pad"]:
            slots[-c["pad"]:] = -1
        s["slots"] = slots
    if c["count"]:
        s["counts"] = torch.tensor(kept(c), dtype=torch.int32, device=dev)


def _prepare_append(c, g, dev, s, rn):
    """Pages in a shuffled order for the positions that are written; the table's other entries are not looked at."""
    B, T, page, Hq, Hk, d = (c[x] for x in ("B", "T", "page", "Hq", "Hk", "d"))
    lens, new = contexts(c), news(c)
    first = torch.tensor([n // page for n in lens])
    need = torch.tensor([(n + m - 1) // page + 1 for n, m in zip(lens, new)]) - first
    total, width = int(need.sum()) + 3, int((first + need).max())
    order = torch.randperm(total, generator=g, device=dev).int()
    at = torch.cat((torch.zeros(1, dtype=torch.int64), need.cumsum(0)))
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    for b in range(B):
        table[b, first[b]:first[b] + need[b]] = order[at[b]:at[b + 1]]
    s["table"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device=dev)
    s["kc"], s["vc"] = (torch.full((total, page, Hk, d), float("nan"), dtype=BF16, device=dev) for _ in "kv")
    rows = (1, T) if c["packed"] else (B, T)
    qkv = rn(*rows, Hq + 2 * Hk, d) * 3   # one projection, of which the call takes its parts
    s["q"] = qkv[:, :, :Hq] if c["queries"] else None
    s["k"], s["v"] = qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:]
    s["wq"], s["wk"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev) for _ in "qk")
    s["cu"] = s["rows"] = s["counts"] = None
    if c["packed"]:
        s["cu"] = torch.cat((torch.zeros(1, dtype=torch.int64), torch.tensor(new).cumsum(0))).int().to(dev)
    if c["pick"]:
        s["counts"] = torch.tensor(kept(c), dtype=torch.int32, device=dev)
        # an increasing choice of rows for each sequence, in its first `counts` entries
        key = torch.rand((B, T), generator=g, device=dev)
        key = torch.where(torch.arange(T, device=dev)[None] < s["counts"][:, None], key.argsort(1), T)
        s["rows"] = key.sort(1).values.clamp_max(T - 1).to(torch.int32)


def _prepare_shared(c, g, dev, s, rn):
    """A cache whose page tables begin with the same pages for the sequences of a group.  Slots never written are NaN."""
    B, T, page, Hk, d = (c[x] for x in ("B", "T", "page", "Hk", "d"))
    mine, groups = contexts(c), members(c)
    whole = [0] * B   # pages of the sequence's prefix
    for b0, n, p in groups:
        whole[b0:b0 + n] = [p // page] * n
    lens = [w * page + m for w, m in zip(whole, mine)]
    need = [-(-(n + T) // page) for n in lens]
    total = sum(p // page for _, _, p in groups) + sum(e - w for e, w in zip(need, whole)) + 3
    order = torch.randperm(total, generator=g, device=dev).int()
    table = torch.full((B, max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b0, n, p in groups:
        table[b0:b0 + n, :p // page] = order[at:at + p // page]
        at += p // page
    for b in range(B):
        table[b, whole[b]:need[b]] = order[at:at + need[b] - whole[b]]
        at += need[b] - whole[b]
    s["kc"], s["vc"] = (torch.randn((total, page, Hk, d), generator=g, device=dev, dtype=BF16) for _ in "kv")
    for b in range(B):   # the rest of the last page, and what no table names
        if need[b] * page > lens[b] + T:
            last = table[b, need[b] - 1:need[b]].long()
            for x in (s["kc"], s["vc"]):
                x[last, (lens[b] + T) % page:] = float("nan")
    for x in (s["kc"], s["vc"]):
        x[order[at:].long()] = float("nan")
    s["table"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device=dev)
    s["cu"] = torch.tensor([b0 for b0, _, _ in groups] + [groups[-1][0] + groups[-1][1]], dtype=torch.int32, device=dev)
    s["shared"] = torch.tensor([p // page * page for _, _, p in groups], dtype=torch.int32, device=dev)
    s["q"] = rn(B, T, c["Hq"], d) * 2
    s["tree"] = _trees(g, B, T, dev) if c["tree"] else None


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 13)
    s = {"case": c}
    rn = lambda *shape: torch.randn(shape, generator=g, device=dev, dtype=BF16)
    {"delta": _prepare_delta, "append": _prepare_append, "shared": _prepare_shared}[c["op"]](c, g, dev, s, rn)
    return s


# ------------------------------------------------------------------ plain forms
def _delta_plain(s):
    """S <- g S + beta k (v - g S^T k)^T, o = S^T q, token by token."""
    c = s["case"]
    live = torch.ones(c["B"], dtype=torch.bool, device=s["q"].device) if s["slots"] is None else s["slots"] >= 0
    at = torch.arange(c["B"], device=s["q"].device) if s["slots"] is None else s["slots"].long()
    at = at[live]
    S = s["state"][at]
    q, k, v, a, beta = (s[x][live].float() for x in ("q", "k", "v", "a", "beta"))
    lam = -torch.log1p(torch.exp(a)) if c["soft"] else BOUND / (1 + torch.exp(-a))
    gate = lam.exp()[..., None, None]
    o = torch.zeros((c["B"], c["T"], c["H"], c["dv"]), device=S.device)
    got = []
    n = None if s["counts"] is None else s["counts"][live].long()
    end = S
    for t in range(c["T"]):
        S = gate[:, t] * S
        e = v[:, t] - (S * k[:, t, :, :, None]).sum(2)
        S = S + (beta[:, t, :, None] * k[:, t])[..., None] * e[:, :, None]
        got.append((S * q[:, t, :, :, None]).sum(2))
        end = S if n is None else torch.where((t < n)[:, None, None, None], S, end)
    o[live] = torch.stack(got, 1)
    s["state"][at] = end
    return o if c["f32"] else o.to(BF16), s["state"]


def _split(x, rot, inter):
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])


def _join(a, b, rest, inter):
    ab = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((ab, rest), -1)


def _norm_plain(x, w, pos, rot, inter):
    """Rows x [.., H, d] at positions pos [..]: RMS norm of every head, then the rotation."""
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    if not rot:
        return y.to(BF16)
    f = BASE ** (-torch.arange(0, rot, 2, device=x.device, dtype=F64) / rot)
    ang = pos.double()[..., None, None] * f
    cos, sin = ang.cos().float(), ang.sin().float()
    a, b = _split(y, rot, inter)
    return _join(a * cos - b * sin, b * cos + a * sin, y[..., rot:], inter).to(BF16)


def _places(s):
    """For every token of k: its sequence, its number among the sequence's new ones, and whether it is written."""
    c, dev = s["case"], s["k"].device
    if s["cu"] is not None:
        t = torch.arange(c["T"], device=dev)
        b = torch.bucketize(t, s["cu"][1:-1].long(), right=True)
        return b[None], (t - s["cu"].long()[b])[None], None
    b = torch.arange(c["B"], device=dev)[:, None].expand(-1, c["T"])
    j = torch.arange(c["T"], device=dev)[None].expand(c["B"], -1)
    return b, j, None if s["counts"] is None else j < s["counts"][:, None]


def _append_plain(s):
    c, page = s["case"], s["case"]["page"]
    b, j, live = _places(s)
    pos = s["lens"].long()[b] + j
    qn = _norm_plain(s["q"], s["wq"], pos, c["rot"], c["inter"]) if c["queries"] else None
    k, v = s["k"], s["v"]
    if s["rows"] is not None:
        pick = s["rows"].long()[..., None, None].expand_as(k)
        k, v = k.gather(1, pick), v.gather(1, pick)
    k = _norm_plain(k, s["wk"], pos, c["rot"], c["inter"])
    slot = s["table"].long()[b, pos // page] * page + pos % page
    if live is not None:
        k, v, slot = k[live], v[live], slot[live]
    s["kc"].view(-1, *k.shape[-2:]).index_copy_(0, slot.reshape(-1), k.reshape(-1, *k.shape[-2:]))
    s["vc"].view(-1, *v.shape[-2:]).index_copy_(0, slot.reshape(-1), v.reshape(-1, *v.shape[-2:]))
    return qn, s["kc"], s["vc"]


def _cached_group(s, b0, b1):
    """Sequences b0 .. b1 - 1, each over all of its own page table: outputs [b, T, Hq, d] and log-sums [b, T, Hq]."""
    c, dev = s["case"], s["q"].device
    T, Hk, d, page = c["T"], c["Hk"], c["d"], c["page"]
    G, n = c["Hq"] // Hk, b1 - b0
    lens = s["lens"][b0:b1].long()
    slot = torch.arange(s["table"].shape[1] * page, device=dev)
    have = slot[None] < lens[:, None] + T
    pages = s["table"][b0:b1].long().clamp_min(0)
    gather = lambda x: x[pages].flatten(1, 2).float().masked_fill(~have[..., None, None], 0)   # [n, S, Hk, d]
    k, v = gather(s["kc"]), gather(s["vc"])
    i, draft = torch.arange(T, device=dev), slot[None] - lens[:, None]
    if s["tree"] is None:
        see = draft[:, None] <= i[None, :, None]
    else:
        bit = (s["tree"][b0:b1][:, :, None] >> draft.clamp(0, 63)[:, None]) & 1
        see = (draft[:, None] < 0) | ((bit == 1) & (draft[:, None] < T))
    see = (see & have[:, None])[:, None, None]                                                   # [n, 1, 1, T, S]
    q = s["q"][b0:b1].reshape(n, T, Hk, G, d).float()
    x = torch.einsum("bnhgd,bshd->bhgns", q, k) * d ** -0.5
    x = x.masked_fill(~see, float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = (x - m.clamp_min(torch.finfo(F32).min)).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgns,bshd->bnhgd", p / torch.where(z > 0, z, 1), v)
    lse = (m + z.log())[..., 0].permute(0, 3, 1, 2)
    return o.reshape(n, T, -1, d), lse.reshape(n, T, -1)


def _shared_plain(s):
    c = s["case"]
    cap = s["table"].shape[1] * c["page"]
    step = max(1, (1 << 31) // (cap * max(c["Hk"] * c["d"], c["Hq"] * c["T"])))
    parts = [_cached_group(s, b, min(c["B"], b + step)) for b in range(0, c["B"], step)]
    return torch.cat([p[0] for p in parts]).to(BF16), torch.cat([p[1] for p in parts])


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s, s["case"])
    return {"delta": _delta_plain, "append": _append_plain, "shared": _shared_plain}[s["case"]["op"]](s)


def _run_own(s, c):
    from chunked_linear_attention_bounded_gb300 import bdla
    if "ws" not in s:
        s["ws"] = bdla.Workspace(256, s["k" if "k" in s else "q"].device)   # kept from call to call, as a program does
    ws = s["ws"]
    if c["op"] == "delta":
        o = bdla.decode_delta(s["q"], s["k"], s["v"], s["a"], s["beta"], s["state"], slots=s["slots"], counts=s["counts"],
                              b=BOUND, mode=bdla.SOFTPLUS if c["soft"] else bdla.BOUNDED, o_dtype=F32 if c["f32"] else BF16,
                              ws=ws)
        return o, s["state"]
    if c["op"] == "append":
        qn = bdla.qk_norm_append(s["q"], s["k"], s["v"], s["wq"] if c["queries"] else None, s["wk"], s["kc"], s["vc"],
                                 s["table"], s["lens"], rows=s["rows"], counts=s["counts"], rotary=c["rot"], base=BASE,
                                 interleaved=c["inter"], cu_seqlens=s["cu"], eps=EPS, ws=ws)
        return qn, s["kc"], s["vc"]
    return bdla.attn_shared(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["cu"], s["shared"], tree=s["tree"], ws=ws)


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    c, s = case, prepare(case, seed)
    return {"delta": _delta_exact, "append": _append_exact, "shared": _shared_exact}[c["op"]](c, s)


def _delta_exact(c, s):
    """S_t = g_t (I - beta_t k_t k_t^T) S_(t-1) + beta_t k_t v_t^T,  o_t = S_t^T q_t, a sequence at a time."""
    B, T, H, dk, dv = (c[x] for x in ("B", "T", "H", "dk", "dv"))
    dev = s["q"].device
    o = torch.zeros((B, T, H, dv), dtype=F64, device=dev)
    state = s["state"].double()
    eye = torch.eye(dk, dtype=F64, device=dev)
    slots = list(range(B)) if s["slots"] is None else s["slots"].tolist()
    counts = kept(c) or [T] * B
    a = s["a"].double()
    g = torch.exp(-torch.nn.functional.softplus(a) if c["soft"] else BOUND * torch.sigmoid(a))
    for b, at in enumerate(slots):
        if at < 0:
            continue
        S = state[at].clone()
        for t in range(T):
            if t == counts[b]:
                state[at] = S
            k, v, q, w = s["k"][b, t].double(), s["v"][b, t].double(), s["q"][b, t].double(), s["beta"][b, t].double()
            A = eye - w[:, None, None] * k[:, :, None] * k[:, None]
            S = g[b, t, :, None, None] * (A @ S) + (w[:, None] * k)[:, :, None] * v[:, None]
            o[b, t] = torch.einsum("hij,hi->hj", S, q)
        if counts[b] == T:
            state[at] = S
    return o, state


def _turned(c, x, w, pos):
    """Rows [n, H, d] at positions [n], normed and turned as complex numbers."""
    u = x.double()
    y = u / ((u ** 2).sum(-1, keepdim=True) / c["d"] + EPS) ** 0.5 * w.double()
    if c["rot"]:
        i = torch.arange(c["rot"] // 2, dtype=F64, device=x.device)
        ang = pos.double()[:, None] / BASE ** (2 * i / c["rot"])
        r = y[..., :c["rot"]]
        r = r.reshape(*r.shape[:-1], -1, 2) if c["inter"] else r.reshape(*r.shape[:-1], 2, -1).transpose(-1, -2)
        z = torch.view_as_complex(r.contiguous()) * torch.polar(torch.ones_like(ang), ang)[:, None]
        r = torch.view_as_real(z)
        y[..., :c["rot"]] = (r if c["inter"] else r.transpose(-1, -2)).flatten(-2)
    return y


def _append_exact(c, s):
    B, T, page = c["B"], c["T"], c["page"]
    lens, new, n_kept = contexts(c), news(c), kept(c)
    dev = s["k"].device
    kc, vc = s["kc"].double(), s["vc"].double()
    qs, at = [], 0
    for b in range(B):
        n = new[b]
        q, k, v = ((None if x is None else x[0, at:at + n] if c["packed"] else x[b]) for x in (s["q"], s["k"], s["v"]))
        at += n
        pos = lens[b] + torch.arange(n, device=dev)
        if q is not None:
            qs.append(_turned(c, q, s["wq"], pos))
        if n_kept is not None:
            pick = s["rows"][b, :n_kept[b]].long()
            if not n_kept[b]:
                continue
            k, v, pos = k[pick], v[pick], pos[:n_kept[b]]
        page_of = s["table"][b].long()[pos // page]
        kc[page_of, pos % page] = _turned(c, k, s["wk"], pos)
        vc[page_of, pos % page] = v.double()
    qn = None if not qs else torch.cat(qs).reshape(s["q"].shape)
    return qn, kc, vc


def _shared_exact(c, s):
    T, Hq, Hk, d, page = c["T"], c["Hq"], c["Hk"], c["d"], c["page"]
    dev = s["q"].device
    o = torch.zeros((c["B"], T, Hq, d), dtype=F64, device=dev)
    lse = torch.full((c["B"], T, Hq), -math.inf, dtype=F64, device=dev)
    table, lens = s["table"].cpu(), s["lens"].tolist()
    tree = s["tree"].cpu() if s["tree"] is not None else None
    for b, n in enumerate(lens):
        used = table[b, :-(-(n + T) // page)].long().to(dev)
        k = s["kc"][used].flatten(0, 1)[:n + T].double().transpose(0, 1)   # [Hk, S, d]
        v = s["vc"][used].flatten(0, 1)[:n + T].double().transpose(0, 1)
        see = torch.ones((T, n + T), dtype=torch.bool)
        for i in range(T):
            for j in range(T):
                see[i, n + j] = j <= i if tree is None else bool((int(tree[b, i]) >> j) & 1)
        see = see.to(dev)[:, None].expand(-1, Hq // Hk, -1).reshape(T * (Hq // Hk), -1)
        some = see.any(1)
        q = s["q"][b].double().reshape(T, Hk, Hq // Hk, d).transpose(0, 1).reshape(Hk, -1, d)
        x = q @ k.transpose(1, 2) / math.sqrt(d)
        x = torch.where(see, x, -math.inf)
        l = torch.logsumexp(x, -1)
        p = torch.where(some[:, None], torch.exp(x - torch.where(some, l, 0.0)[..., None]), 0.0)
        back = lambda y: y.reshape(Hk, T, Hq // Hk, -1).transpose(0, 1).reshape(T, Hq, -1)
        o[b], lse[b] = back(p @ v), back(l)[..., 0]
    return o, lse


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    B, T = c["B"], c["T"]
    if c["op"] == "delta":
        used, el = B - c["pad"], c["H"] * c["dk"] * c["dv"]
        rows = used * T * c["H"] * (4 * c["dk"] + 2 * c["dv"] + 8)
        out = B * T * c["H"] * c["dv"] * (4 if c["f32"] else 2)
        writes = used if not c["count"] else sum(n > 0 for n in kept(c)[:used])
        # a token: the read S^T k, the update, the read S^T q, two operations an element each
        return {"bytes": (used + writes) * el * 4 + rows + out, "flops": used * T * el * 6}
    d, Hq, Hk = c["d"], c["Hq"], c["Hk"]
    if c["op"] == "append":
        tokens = c["T"] if c["packed"] else B * T
        rows = tokens if not c["pick"] else sum(kept(c))
        el = (tokens * Hq if c["queries"] else 0) + rows * Hk
        return {"bytes": (el + rows * Hk) * d * 4, "flops": el * d * 7}
    lens, groups = contexts(c), members(c)
    once = sum(p // c["page"] * c["page"] for _, _, p in groups)
    pairs = sum(n * (p // c["page"] * c["page"]) for _, n, p in groups) + sum(lens) + B * T
    keys = once + sum(lens) + B * T
    return {"bytes": keys * Hk * d * 4 + 2 * B * T * Hq * d * 2, "flops": pairs * T * Hq * d * 4}
