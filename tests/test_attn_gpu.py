"""The softmax layer's kernels against the 64-bit references of _attn_ref, with that module's derived tolerances."""
import math

import pytest
import torch

import _attn_ref as ref
from chunked_linear_attention_bounded_gb300 import bdla

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(BF16)


def _cu(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ norm and rotation
NORM = [
    # B, T, lens, Hq, Hk, d, rotary, interleaved, far
    (1, 1, None, 1, 1, 128, 128, False, 0),
    (1, 1, None, 32, 8, 128, 128, False, 1 << 30),
    (3, 1, None, 5, 5, 64, 48, True, 1000000),
    (2, 77, None, 3, 1, 64, 64, False, 0),
    (1, 130, (1, 0, 100, 29), 6, 2, 128, 32, True, 0),
    (1, 300, (7, 293), 4, 4, 128, 96, False, 0),
    (1, 40, None, 2, 2, 64, 0, False, 0),
    (1, 9001, (4000, 5001), 4, 2, 64, 16, False, 0),
]


@pytest.mark.parametrize("case", NORM, ids=lambda c: "-".join(str(x) for x in c))
def test_norm_and_gradient(case):
    B, T, lens, Hq, Hk, d, rot, inter, far = case
    g = _gen(T + d + rot)
    qkv = _rn(g, B, T, Hq + 2 * Hk, d) * 2           # views of one projection
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    wq, wk = (1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    cu = _cu(lens) if lens else None
    pos = torch.randint(far // 2, far, (B, T), generator=g, device="cuda", dtype=torch.int32) if far else None
    kw = dict(rotary=rot, base=10000.0, interleaved=inter, positions=pos, cu_seqlens=cu, eps=1e-5)
    where = pos.double() if far else ref.positions(B, T, cu, "cuda")
    qn, kn = bdla.qk_norm(q, k, wq, wk, **kw)
    for gdt in (BF16, torch.float32):
        dqn, dkn = _rn(g, B, T, Hq, d).to(gdt), _rn(g, B, T, Hk, d).to(gdt)
        dq, dk, dwq, dwk = bdla.qk_norm_bwd(q, k, wq, wk, dqn, dkn, **kw)
        for t0 in range(0, T, 1500):   # the reference's rotations are d x d a token
            sl = slice(t0, min(T, t0 + 1500))
            R = ref.rotation(where[:, sl], rot, 10000.0, d, inter)
            ref.check("qn", qn[:, sl], ref.norm(q[:, sl], wq, R, 1e-5))
            ref.check("kn", kn[:, sl], ref.norm(k[:, sl], wk, R, 1e-5))
            a, b = ref.norm(q[:, sl], wq, R, 1e-5, dqn[:, sl]), ref.norm(k[:, sl], wk, R, 1e-5, dkn[:, sl])
            ref.check("dq", dq[:, sl], a[0])
            ref.check("dk", dk[:, sl], b[0])
            sums = [(a[1], b[1])] if t0 == 0 else sums + [(a[1], b[1])]
        for i, (n, x) in enumerate((("dwq", dwq), ("dwk", dwk))):
            ref.check(n, x, (sum(s[i][0] for s in sums), sum(s[i][1] for s in sums)))
        again = bdla.qk_norm_bwd(q, k, wq, wk, dqn, dkn, **kw)
        assert all(torch.equal(x, y) for x, y in zip((dq, dk, dwq, dwk), again))


# more tokens than the gradient's lanes hold at a time, so that each walks several; heads that leave a turn half empty
@pytest.mark.parametrize("case", [(1, 130000, (70001, 59999), 1, 1, 64, 32, True, 0), (2, 30011, None, 3, 3, 128, 128, False, 0)],
                         ids=lambda c: "-".join(str(x) for x in c))
def test_norm_gradient_of_many_tokens(case):
    test_norm_and_gradient(case)


def test_norm_gradient_on_another_stream_and_in_a_graph():
    g = _gen(12)
    q, k, dqn, dkn = _rn(g, 1, 5000, 4, 64), _rn(g, 1, 5000, 2, 64), _rn(g, 1, 5000, 4, 64), _rn(g, 1, 5000, 2, 64)
    w = 1 + 0.3 * torch.randn(64, generator=g, device="cuda")
    want = bdla.qk_norm_bwd(q, k, w, w, dqn, dkn)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = bdla.qk_norm_bwd(q, k, w, w, dqn, dkn, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    ws = bdla.Workspace(1 << 22, "cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = bdla.qk_norm_bwd(q, k, w, w, dqn, dkn, ws=ws)
    for x in got:
        x.fill_(7)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_norm_of_no_tokens():
    q = torch.empty((1, 0, 4, 64), dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    qn, kn = bdla.qk_norm(q, q, w, w)
    assert qn.shape == q.shape
    _, _, dwq, dwk = bdla.qk_norm_bwd(q, q, w, w, q, q)
    assert float(dwq.abs().sum() + dwk.abs().sum()) == 0.0


def test_norm_makes_the_unit_keys_of_the_linear_attention():
    g = _gen(3)
    q, k = _rn(g, 1, 50, 2, 128), _rn(g, 1, 50, 2, 128)
    w = torch.full((128,), 128 ** -0.5, device="cuda")
    _, kn = bdla.qk_norm(q, k, w, w, rotary=0, eps=0.0)
    want = k.double() / k.double().norm(dim=-1, keepdim=True)
    ref.check("kn", kn, (want, 2.0 ** -8 * want.abs() + 2.0 ** -18))


# ------------------------------------------------------------------ whole documents
ATTN = [
    # B, T, lens, Hq, Hk, d, spread of the logits
    (1, 1, None, 1, 1, 64, 1),
    (2, 3, None, 2, 1, 128, 1),
    (1, 127, None, 3, 1, 64, 2),
    (1, 128, None, 2, 2, 128, 1),
    (3, 129, None, 8, 1, 64, 1),
    (1, 256, None, 4, 2, 128, 6),
    (2, 257, None, 5, 5, 128, 1),
    (1, 385, None, 2, 1, 64, 30),
    (1, 900, (1, 0, 128, 0, 257, 129, 1, 384), 6, 2, 128, 1),
    (1, 900, (300, 299, 301), 4, 4, 64, 3),
    (1, 2100, (2100,), 3, 1, 128, 1),
    (1, 3001, (1000, 2001), 8, 2, 64, 1),
]


def _attn_inputs(case, seed=0):
    B, T, lens, Hq, Hk, d, spread = case
    g = _gen(T * 3 + Hq + d + seed)
    q, k, v, dO = _rn(g, B, T, Hq, d) * spread, _rn(g, B, T, Hk, d), _rn(g, B, T, Hk, d), _rn(g, B, T, Hq, d)
    return q, k, v, dO, _cu(lens) if lens else None


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(str(x) for x in c))
def test_attn_forward(case):
    q, k, v, _, cu = _attn_inputs(case)
    ws = bdla.Workspace(256, "cuda")
    o, lse = bdla.attn_fwd(q, k, v, cu_seqlens=cu, ws=ws)
    assert ws.read_device_status() == bdla.OK
    want = ref.attn(q, k, v, case[5] ** -0.5, cu)
    ref.check("o", o, want["o"])
    ref.check("lse", lse, want["lse"])


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(str(x) for x in c))
def test_attn_gradient(case):
    q, k, v, dO, cu = _attn_inputs(case, seed=1)
    scale = case[5] ** -0.5
    want = ref.attn(q, k, v, scale, cu, dO)
    o, lse = want["o"][0].to(BF16), want["lse"][0].float()
    ws = bdla.Workspace(256, "cuda")
    got = bdla.attn_bwd(q, k, v, o, lse, dO, cu_seqlens=cu, ws=ws)
    assert ws.read_device_status() == bdla.OK
    for n, x in zip(("dq", "dk", "dv"), got):
        ref.check(n, x, want[n])
    again = bdla.attn_bwd(q, k, v, o, lse, dO, cu_seqlens=cu, ws=ws)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


def test_attn_gradient_against_differences():
    """The kernels' gradient along a direction is the difference quotient of the 64-bit loss, within the sum of its
    entries' tolerances; the kernels' own forward feeds it."""
    q, k, v, dO, cu = _attn_inputs((1, 200, (60, 140), 4, 2, 64, 1), seed=2)
    o, lse = bdla.attn_fwd(q, k, v, scale=0.2, cu_seqlens=cu)
    got = bdla.attn_bwd(q, k, v, o, lse, dO, scale=0.2, cu_seqlens=cu)
    tol = ref.attn(q, k, v, 0.2, cu, dO)
    base = [x.double() for x in (q, k, v)]
    for i, n in enumerate(("dq", "dk", "dv")):
        u = torch.randn(base[i].shape, generator=_gen(i), device="cuda", dtype=torch.float64)
        loss = lambda e: (ref.attn(*[x + (e * u if j == i else 0) for j, x in enumerate(base)], 0.2, cu)["o"][0] * dO).sum()
        diff = (loss(1e-4) - loss(-1e-4)) / 2e-4
        # twice the tolerance: o and lse carry the forward kernel's own error here
        assert abs(float((got[i].double() * u).sum() - diff)) <= float((2 * tol[n][1] * u.abs()).sum()) + 1e-5 * abs(float(diff))


@pytest.mark.parametrize("d", [64, 128])
def test_attn_first_tokens_have_no_score_gradient(d):
    """A token that sees itself alone has ds = p (dp - delta) = 0: its dq, and the dk of a document of one token, are
    zero to the bit, as the difference of equal numbers is."""
    lens = (1, 1, 3, 1, 200, 1, 129)
    q, k, v, dO, cu = _attn_inputs((1, sum(lens), lens, 6, 2, d, 2), seed=6)
    o, lse = bdla.attn_fwd(q, k, v, cu_seqlens=cu)
    dq, dk, dv = bdla.attn_bwd(q, k, v, o, lse, dO, cu_seqlens=cu)
    at = 0
    for n in lens:
        assert float(dq[0, at].abs().max()) == 0.0
        if n == 1:
            assert float(dk[0, at].abs().max()) == 0.0
        at += n


def test_attn_rows_whose_maximum_keeps_growing():
    """Scores that rise along the keys, so that every tile raises the running maximum, up to far beyond e^88."""
    T, d = 700, 64
    g = _gen(5)
    q = torch.ones((1, T, 2, d), device="cuda").to(BF16)
    k = (torch.arange(T, device="cuda")[None, :, None, None] / 64 + 0.1 * torch.randn((1, T, 1, d), generator=g, device="cuda")).to(BF16)
    v, dO = _rn(g, 1, T, 1, d), _rn(g, 1, T, 2, d)
    for sign in (1, -1):
        o, lse = bdla.attn_fwd(sign * q, k, v, scale=1.0)
        want = ref.attn(sign * q, k, v, 1.0, None, dO)
        ref.check("o", o, want["o"])
        ref.check("lse", lse, want["lse"])
        got = bdla.attn_bwd(sign * q, k, v, want["o"][0].to(BF16), want["lse"][0].float(), dO, scale=1.0)
        # lse rounds to fp32 at a size of several hundred: every p is off by up to its step there
        step = float(want["lse"][0].abs().max()) * 2.0 ** -23
        for n, x in zip(("dq", "dk", "dv"), got):
            ref.check(n, x, (want[n][0], want[n][1] * (1 + step / ref.H)))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attn_documents_do_not_reach_each_other(bad):
    """A document of infinities or NaN between two others changes nothing in them."""
    lens = (100, 90, 200)
    q, k, v, dO, cu = _attn_inputs((1, 390, lens, 4, 2, 128, 1), seed=3)
    o, lse = bdla.attn_fwd(q, k, v, cu_seqlens=cu)
    clean = bdla.attn_bwd(q, k, v, o, lse, dO, cu_seqlens=cu)
    for x in (q, k, v, dO):
        x[:, 100:190] = bad
    o2, lse2 = bdla.attn_fwd(q, k, v, cu_seqlens=cu)
    o3 = o.clone()
    o3[:, 100:190] = bad
    dirty = bdla.attn_bwd(q, k, v, o3, lse2, dO, cu_seqlens=cu)
    for x, y in [(o, o2)] + list(zip(clean, dirty)):
        assert torch.equal(x[:, :100], y[:, :100]) and torch.equal(x[:, 190:], y[:, 190:])
    assert torch.equal(lse[:, :100], lse2[:, :100]) and torch.equal(lse[:, 190:], lse2[:, 190:])


def test_attn_malformed_offsets_are_reported():
    q, k, v, dO, _ = _attn_inputs((1, 300, None, 2, 1, 64, 1))
    for offs in ([0, 200, 100, 300], [0, 100, 400], [5, 100, 300], [0, 100, 299], [-7, 100, 300]):
        cu = torch.tensor(offs, dtype=torch.int32, device="cuda")
        ws = bdla.Workspace(256, "cuda")
        o, lse = bdla.attn_fwd(q, k, v, cu_seqlens=cu, ws=ws)
        assert ws.read_device_status() == bdla.ERR_DEVICE
        bdla.attn_bwd(q, k, v, torch.zeros_like(q), torch.zeros_like(lse), dO, cu_seqlens=cu, ws=ws)
        assert ws.read_device_status() == bdla.ERR_DEVICE
    o, lse = bdla.attn_fwd(q, k, v)
    ref.check("o", o, ref.attn(q, k, v, 0.125)["o"])


def test_attn_of_no_tokens():
    q = torch.empty((1, 0, 4, 64), dtype=BF16, device="cuda")
    o, lse = bdla.attn_fwd(q, q, q, cu_seqlens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert o.shape == q.shape and lse.shape == (4, 0)
    assert all(x.shape == q.shape for x in bdla.attn_bwd(q, q, q, o, lse, q))


def test_attn_on_another_stream_and_in_a_graph():
    q, k, v, dO, cu = _attn_inputs((1, 700, (500, 200), 4, 2, 128, 1), seed=4)
    o, lse = bdla.attn_fwd(q, k, v, cu_seqlens=cu)
    grads = bdla.attn_bwd(q, k, v, o, lse, dO, cu_seqlens=cu)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, lse2 = bdla.attn_fwd(q, k, v, cu_seqlens=cu, stream=side)
    grads2 = bdla.attn_bwd(q, k, v, o2, lse2, dO, cu_seqlens=cu, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and all(torch.equal(x, y) for x, y in zip(grads, grads2))
    ws = bdla.Workspace(1 << 20, "cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, lse3 = bdla.attn_fwd(q, k, v, cu_seqlens=cu, ws=ws)
        grads3 = bdla.attn_bwd(q, k, v, o3, lse3, dO, cu_seqlens=cu, ws=ws)
    v.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    ref.check("o", o3, ref.attn(q, k, v, 128 ** -0.5, cu)["o"])
    ref.check("lse", lse3, ref.attn(q, k, v, 128 ** -0.5, cu)["lse"])
    assert torch.equal(grads3[2], grads[2])   # dv does not depend on v


# ------------------------------------------------------------------ the paged cache
def _pool(g, lens, T, page, Hk, d, spare=2):
    """A cache whose every slot is NaN, a page table in a shuffled order, and the sequences' own rows."""
    need = [-(-(n + T) // page) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=g, device="cuda")
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].int()
        at += n
    kc = torch.full((sum(need) + spare, page, Hk, d), float("nan"), dtype=BF16, device="cuda")
    return kc, kc.clone(), table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def _fill(kc, vc, table, b, upto, g):
    page = kc.shape[1]
    if upto == 0:
        return
    t = torch.arange(upto, device="cuda")
    p = table[b].long()[t // page]
    kc[p, t % page] = _rn(g, upto, *kc.shape[2:])
    vc[p, t % page] = _rn(g, upto, *kc.shape[2:])


APPEND = [((0,), 1, 16, 1, 64), ((5, 0, 31), 7, 8, 2, 128), ((3, 90), 50, 24, 8, 128), ((2, 1, 0, 9), 3, 1, 3, 64),
          ((100,), 300, 100, 1, 128)]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(x) for x in c))
def test_append_writes_its_rows_and_nothing_else(case):
    lens, T, page, Hk, d = case
    g = _gen(T + page)
    kc, vc, table, dl = _pool(g, lens, T, page, Hk, d)
    B = len(lens)
    k, v = _rn(g, B, T, Hk, d), _rn(g, B, T, Hk, d)
    for pick in (False, True):
        rows = torch.randint(0, T, (B, T), generator=g, device="cuda", dtype=torch.int32) if pick else None
        counts = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if pick else None
        want_k, want_v = kc.clone(), vc.clone()
        for b in range(B):
            for j in range(int(counts[b]) if pick else T):
                t, src = lens[b] + j, int(rows[b, j]) if pick else j
                want_k[int(table[b, t // page]), t % page] = k[b, src]
                want_v[int(table[b, t // page]), t % page] = v[b, src]
        ws = bdla.Workspace(256, "cuda")
        bdla.cache_append(k, v, kc, vc, table, dl, rows=rows, counts=counts, ws=ws)
        assert ws.read_device_status() == bdla.OK
        assert torch.equal(kc.view(torch.int16), want_k.view(torch.int16))
        assert torch.equal(vc.view(torch.int16), want_v.view(torch.int16))


def test_append_reports_what_it_cannot_write():
    g = _gen(8)
    k = _rn(g, 2, 4, 2, 64)
    for what in ("page", "table", "row", "count", "negative count", "len"):
        kc, vc, table, lens = _pool(g, (3, 5), 4, 4, 2, 64)
        rows = torch.arange(4, device="cuda", dtype=torch.int32).repeat(2, 1)
        counts = torch.full((2,), 4, dtype=torch.int32, device="cuda")
        if what == "page":
            table[1, 1] = kc.shape[0]
        elif what == "table":
            lens[1] = table.shape[1] * 4 - 2
        elif what == "row":
            rows[1, 2] = 4
        elif what == "count":
            counts[0] = 5
        elif what == "negative count":
            counts[0] = -1
        else:
            lens[0] = -2
        ws = bdla.Workspace(256, "cuda")
        bdla.cache_append(k, k, kc, vc, table, lens, rows=rows, counts=counts, ws=ws)
        assert ws.read_device_status() == bdla.ERR_DEVICE, what


def _tree(g, B, T):
    bits = torch.zeros((B, T), dtype=torch.int64)
    r = torch.rand((B, T), generator=g, device="cuda").cpu()
    for b in range(B):
        for i in range(T):
            par = int(r[b, i] * (i + 1)) - 1
            bits[b, i] = (bits[b, par] if par >= 0 else 0) | ((1 << i) if i < 63 else -(1 << 63))
    return bits.cuda()


CACHED = [
    # lens, T, page, Hq, Hk, d, tree
    ((0,), 1, 16, 1, 1, 64, False),
    ((0, 1, 2, 63, 64, 65), 1, 16, 8, 2, 128, False),
    ((127, 128, 129, 500), 1, 24, 3, 1, 64, False),
    ((1000, 7), 1, 1, 16, 1, 128, False),
    ((300, 0, 77), 4, 100, 6, 2, 128, False),
    ((200, 0, 511), 5, 8, 4, 4, 64, True),
    ((333, 0), 17, 32, 8, 2, 128, True),
    ((1500, 0, 64), 64, 64, 4, 2, 128, True),
    ((90, 1000), 33, 256, 24, 3, 64, True),
    ((20000,), 1, 64, 8, 1, 128, False),
    ((9000, 10), 3, 48, 2, 2, 64, True),
]


@pytest.mark.parametrize("case", CACHED, ids=lambda c: "-".join(str(x) for x in c))
def test_attn_cached(case):
    lens, T, page, Hq, Hk, d, tree = case
    g = _gen(sum(lens) + T + page)
    kc, vc, table, dl = _pool(g, lens, T, page, Hk, d)
    for b, n in enumerate(lens):
        _fill(kc, vc, table, b, n, g)
    B = len(lens)
    q, k, v = _rn(g, B, T, Hq, d) * 2, _rn(g, B, T, Hk, d), _rn(g, B, T, Hk, d)
    ws = bdla.Workspace(256, "cuda")
    bdla.cache_append(k, v, kc, vc, table, dl, ws=ws)
    bits = _tree(g, B, T) if tree else None
    if tree:
        bits[:, T // 2] = 0                     # sees the context alone, or nothing at all
        bits[-1, 0] = -1                        # bits past the new tokens say nothing
        bits[0, T - 1] = 1
    o, lse = bdla.attn_cached(q, kc, vc, table, dl, tree=bits, scale=0.09, ws=ws)
    assert ws.read_device_status() == bdla.OK
    want_o, want_l = ref.cached(q, kc, vc, table, lens, bits, 0.09)
    ref.check("o", o, want_o)
    ref.check("lse", lse, want_l)
    again = bdla.attn_cached(q, kc, vc, table, dl, tree=bits, scale=0.09, ws=ws)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_cached_sequences_share_pages():
    """Two sequences over the same pages of a common prompt, as after a fork."""
    g = _gen(12)
    kc, vc, table, lens = _pool(g, (64, 64), 1, 32, 2, 128)
    table[1, :2] = table[0, :2]
    _fill(kc, vc, table, 0, 64, g)
    k, q = _rn(g, 2, 1, 2, 128), _rn(g, 2, 1, 4, 128)
    bdla.cache_append(k, k, kc, vc, table, lens)
    (wo, wl) = ref.cached(q, kc, vc, table, [64, 64], None, 0.1)
    o, lse = bdla.attn_cached(q, kc, vc, table, lens, scale=0.1)
    ref.check("o", o, wo)
    ref.check("lse", lse, wl)


def test_cached_reports_pages_it_cannot_read():
    """A bad page, a table that is too short, a negative length: reported, and not seen."""
    g = _gen(14)
    for what in ("page", "negative page", "table", "len"):
        kc, vc, table, lens = _pool(g, (40, 50), 2, 16, 2, 64)
        n = [40, 50]
        for b in range(2):
            _fill(kc, vc, table, b, n[b] + 2, g)
        if what == "page":
            table[1, 1] = kc.shape[0]
        elif what == "negative page":
            table[1, 2] = -5
        elif what == "table":
            table = table[:, :3].contiguous()
            n[1] = 50
        else:
            n[0] = -3
        lens = torch.tensor(n, dtype=torch.int32, device="cuda")
        ws = bdla.Workspace(256, "cuda")
        q = _rn(g, 2, 2, 4, 64)
        o, lse = bdla.attn_cached(q, kc, vc, table, lens, scale=0.1, ws=ws)
        assert ws.read_device_status() == bdla.ERR_DEVICE, what
        want_o, want_l = ref.cached(q, kc, vc, table, n, None, 0.1)
        ref.check("o " + what, o, want_o)
        ref.check("lse " + what, lse, want_l)


@pytest.mark.parametrize("T,Hq", [(1, 4), (20, 4)])
def test_a_cache_without_pages_or_a_table_without_entries(T, Hq):
    """Positions that no page holds: reported, seen by nobody; nothing at all in sequences of length 0 - T."""
    q = _rn(_gen(15), 2, T, Hq, 64)
    lens = torch.tensor([0, 7], dtype=torch.int32, device="cuda")
    empty = torch.empty((0, 16, 2, 64), dtype=BF16, device="cuda")
    some = torch.zeros((3, 16, 2, 64), dtype=BF16, device="cuda")
    for cache, table in ((empty, torch.zeros((2, 3), dtype=torch.int32, device="cuda")),
                         (some, torch.zeros((2, 0), dtype=torch.int32, device="cuda"))):
        ws = bdla.Workspace(256, "cuda")
        o, lse = bdla.attn_cached(q, cache, cache, table, lens, ws=ws)
        assert ws.read_device_status() == bdla.ERR_DEVICE
        assert float(o.float().abs().sum()) == 0.0 and bool((lse == -math.inf).all())


def test_cache_offsets_past_32_bits():
    """Pages whose first element lies past 2^31 (and, in bytes, 2^32)."""
    page, Hk, d = 64, 4, 128
    n_pages = (1 << 31) // (page * Hk * d) + 5
    kc = torch.empty((n_pages, page, Hk, d), dtype=BF16, device="cuda")
    vc = torch.empty_like(kc)
    g = _gen(20)
    table = torch.tensor([[n_pages - 1, n_pages - 3, n_pages - 2]], dtype=torch.int32, device="cuda")
    T = 60
    k, v, q = _rn(g, 1, 130, Hk, d), _rn(g, 1, 130, Hk, d), _rn(g, 1, T, 8, d)
    bdla.cache_append(k, v, kc, vc, table, torch.zeros(1, dtype=torch.int32, device="cuda"))
    lens = torch.tensor([130 - T], dtype=torch.int32, device="cuda")
    o, lse = bdla.attn_cached(q, kc, vc, table, lens)
    used = table[0].long()
    small_k, small_v = kc[used], vc[used]
    local = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    want_o, want_l = ref.cached(q, small_k, small_v, local, [130 - T], None, d ** -0.5)
    ref.check("o", o, want_o)
    ref.check("lse", lse, want_l)


def test_cached_in_a_graph_follows_its_lengths():
    """A captured decode step reads the lengths and the table at replay."""
    g = _gen(21)
    kc, vc, table, lens = _pool(g, (300, 20), 40, 16, 2, 128)
    for b, n in enumerate((340, 60)):
        _fill(kc, vc, table, b, n, g)
    q = _rn(g, 2, 1, 8, 128)
    need = bdla.lib().bdla_workspace_bytes_attn(bdla.ATTN_CACHED, bdla.AttnDims(2, 1, 8, 2, 128), 0, table.shape[1] * 16)
    ws = bdla.Workspace(need, "cuda")
    bdla.attn_cached(q, kc, vc, table, lens, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = bdla.attn_cached(q, kc, vc, table, lens, ws=ws)
    for step in range(3):
        lens.add_(13)
        graph.replay()
        torch.cuda.synchronize()
        n = [300 + 13 * (step + 1), 20 + 13 * (step + 1)]
        want_o, want_l = ref.cached(q, kc, vc, table, n, None, 128 ** -0.5)
        ref.check("o", o, want_o)
        ref.check("lse", lse, want_l)


def test_prompt_then_drafts_then_compaction_agree_with_the_whole_prompt():
    """Norm, whole-prompt attention and the cache together: a prompt, a tree whose accepted path is compacted, and the
    next token give what whole-sequence attention gives."""
    g = _gen(30)
    n, Hq, Hk, d, page = 150, 4, 2, 128, 16
    path = [0, 2, 3]                                   # accepted drafts of six
    wq = wk = torch.ones(d, device="cuda")
    raw_q, raw_k, v = _rn(g, 1, n + 7, Hq, d), _rn(g, 1, n + 7, Hk, d), _rn(g, 1, n + 7, Hk, d)
    # the six drafts' depths: two chains from the context, 0-2-3 and 0-1, and 4-5
    depth = torch.tensor([[0, 1, 1, 2, 0, 1]], device="cuda")
    pos = torch.cat([torch.arange(n, device="cuda")[None], n + depth, torch.tensor([[n + 3]], device="cuda")], 1).int()
    qn, kn = bdla.qk_norm(raw_q, raw_k, wq, wk, positions=pos)
    tree = torch.tensor([[0b1, 0b11, 0b101, 0b1101, 0b10000, 0b110000]], dtype=torch.int64, device="cuda")
    kc, vc, table, lens = _pool(g, (0,), n + 20, page, Hk, d)
    bdla.cache_append(kn[:, :n].contiguous(), v[:, :n].contiguous(), kc, vc, table, lens)
    lens.fill_(n)
    dk, dv = kn[:, n:n + 6].contiguous(), v[:, n:n + 6].contiguous()
    bdla.cache_append(dk, dv, kc, vc, table, lens)
    o, _ = bdla.attn_cached(qn[:, n:n + 6].contiguous(), kc, vc, table, lens, tree=tree)
    rows = torch.tensor([path + [0, 0, 0]], dtype=torch.int32, device="cuda")
    bdla.cache_append(dk, dv, kc, vc, table, lens, rows=rows, counts=torch.tensor([3], dtype=torch.int32, device="cuda"))
    lens.fill_(n + 3)
    bdla.cache_append(kn[:, n + 6:].contiguous(), v[:, n + 6:].contiguous(), kc, vc, table, lens)
    last, _ = bdla.attn_cached(qn[:, n + 6:].contiguous(), kc, vc, table, lens)
    keep = list(range(n)) + [n + p for p in path] + [n + 6]
    whole = [x[:, keep].contiguous() for x in (qn, kn, v)]
    want = ref.attn(*whole, d ** -0.5)["o"]
    ref.check("accepted", o[:, path], tuple(x[:, n:n + 3] for x in want))
    ref.check("next", last, tuple(x[:, n + 3:] for x in want))
    full, _ = bdla.attn_fwd(*whole)
    ref.check("whole", full, want)
