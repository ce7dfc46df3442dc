"""Norm, rotation and append in one call: the bits of the two calls that it stands for, the definition in 64 bits, and the
calls that it has to refuse or record."""
import pytest
import torch

import _attn_ref as ref
from chunked_linear_attention_bounded_gb300 import bdla

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


def _case(B, T, Hq, Hk, d, page, lens, news=None, seed=1, spare=3, views=True):
    """One projection of all new tokens, weights, and a cache with pages in a shuffled order, filled with NaN."""
    g = torch.Generator("cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    qkv = (rn(B, T, Hq + 2 * Hk, d) * 2).to(BF16)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:]
    if not views:
        q, k, v = (x.contiguous() for x in (q, k, v))
    news = [T] * len(lens) if news is None else news
    width = max((n + m - 1) // page + 1 if n + m else 1 for n, m in zip(lens, news)) + 1
    total = len(lens) * width + spare
    order = torch.randperm(total, generator=g, device="cuda").to(I32)
    c = dict(kc=torch.full((total, page, Hk, d), float("nan"), dtype=BF16, device="cuda"),
             vc=torch.full((total, page, Hk, d), float("nan"), dtype=BF16, device="cuda"),
             pages=order[:len(lens) * width].view(len(lens), width).contiguous(),
             lens=torch.tensor(lens, dtype=I32, device="cuda"))
    return q, k, v, 1 + 0.3 * rn(d), 1 + 0.3 * rn(d), c


def _same(x, y):
    return torch.equal(x.view(torch.int16), y.view(torch.int16))   # NaN and all


def _append(q, k, v, wq, wk, c, **kw):
    kc, vc, ws = c["kc"].clone(), c["vc"].clone(), bdla.Workspace(256, "cuda")
    qn = bdla.qk_norm_append(q, k, v, wq, wk, kc, vc, c["pages"], c["lens"], ws=ws, **kw)
    return qn, kc, vc, ws.read_device_status()


CASES = [  # B, T, Hq, Hk, d, page, rotary, interleaved, views
    (1, 1, 1, 1, 64, 16, 64, False, True), (1, 1, 32, 8, 128, 64, 128, False, True), (5, 1, 6, 2, 64, 1, 32, True, False),
    (3, 17, 4, 4, 128, 24, 16, True, True), (2, 300, 16, 2, 128, 48, 0, False, True), (7, 33, 3, 1, 64, 100, 48, False, False),
    (1, 3000, 24, 8, 64, 256, 64, True, True)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_the_bits_of_norm_and_append(case):
    B, T, Hq, Hk, d, page, rot, inter, views = case
    lens = [(37 * b * b + 5 * b) % 700 for b in range(B)]
    q, k, v, wq, wk, c = _case(B, T, Hq, Hk, d, page, lens, views=views)
    kw = dict(rotary=rot, interleaved=inter, base=5000.0, eps=1e-5)
    qn, kc, vc, status = _append(q, k, v, wq, wk, c, **kw)
    pos = c["lens"][:, None] + torch.arange(T, dtype=I32, device="cuda")[None]
    want_q, want_k = bdla.qk_norm(q, k, wq, wk, positions=pos, **kw)
    want_kc, want_vc = c["kc"].clone(), c["vc"].clone()
    bdla.cache_append(want_k, v.contiguous(), want_kc, want_vc, c["pages"], c["lens"])
    assert status == bdla.OK
    assert _same(qn, want_q) and _same(kc, want_kc) and _same(vc, want_vc)
    # the definition
    R = ref.rotation(pos.double(), rot, 5000.0, d, inter)
    ref.check("q", qn, ref.norm(q, wq, R, 1e-5))
    at = (c["pages"].long().gather(1, pos.long() // page), pos.long() % page)
    ref.check("k", kc[at], ref.norm(k, wk, R, 1e-5))
    assert torch.equal(vc[at], v)
    # keys and values alone
    none, kc2, vc2, status = _append(None, k, v, None, wk, c, **kw)
    assert none is None and status == bdla.OK and _same(kc2, want_kc) and _same(vc2, want_vc)


@pytest.mark.parametrize("news", [[1], [0, 5, 0, 1, 300, 1, 0], [1] * 40, [700, 13]])
@pytest.mark.parametrize("d", [64, 128])
def test_packed_tokens_of_all_sequences(news, d):
    lens = [(91 * b) % 130 for b in range(len(news))]
    T = sum(news)
    q, k, v, wq, wk, c = _case(1, T, 4, 2, d, 16, lens, news=news, seed=2)
    cu = torch.tensor([sum(news[:i]) for i in range(len(news) + 1)], dtype=I32, device="cuda")
    qn, kc, vc, status = _append(q, k, v, wq, wk, c, cu_seqlens=cu)
    assert status == bdla.OK
    want_kc, want_vc = c["kc"].clone(), c["vc"].clone()
    for b, n in enumerate(news):
        if n == 0:
            continue
        at = slice(int(cu[b]), int(cu[b + 1]))
        pos = (lens[b] + torch.arange(n, dtype=I32, device="cuda"))[None].contiguous()
        wq_, wk_ = bdla.qk_norm(q[:, at], k[:, at], wq, wk, positions=pos)
        assert _same(qn[:, at], wq_), b
        bdla.cache_append(wk_, v[:, at].contiguous(), want_kc, want_vc, c["pages"][b:b + 1], c["lens"][b:b + 1])
    assert _same(kc, want_kc) and _same(vc, want_vc)


@pytest.mark.parametrize("given", [False, True])
def test_chosen_rows_and_counts(given):
    """The accepted drafts of a tree: their own positions (depths), or those of the places that they take."""
    B, T, lens = 6, 11, [0, 3, 40, 16, 15, 100]
    q, k, v, wq, wk, c = _case(B, T, 6, 3, 128, 16, lens, seed=3)
    g = torch.Generator().manual_seed(4)
    rows = torch.stack([torch.randperm(T, generator=g) for _ in range(B)]).to(I32).cuda()
    counts = torch.tensor([0, 11, 4, 1, 7, 2], dtype=I32, device="cuda")
    own = torch.randint(0, 2000, (B, T), generator=g).to(I32).cuda() if given else None
    qn, kc, vc, status = _append(q, k, v, wq, wk, c, rows=rows, counts=counts, positions=own)
    assert status == bdla.OK
    place = c["lens"][:, None] + torch.arange(T, dtype=I32, device="cuda")[None]
    pick = rows.long()[..., None, None].expand(-1, -1, 3, 128)
    want_q, _ = bdla.qk_norm(q, k, wq, wk, positions=place if own is None else own)
    _, want_k = bdla.qk_norm(q, k.gather(1, pick), wq, wk, positions=place if own is None else own.gather(1, rows.long()))
    want_kc, want_vc = c["kc"].clone(), c["vc"].clone()
    bdla.cache_append(want_k, v.gather(1, pick), want_kc, want_vc, c["pages"], c["lens"], counts=counts)
    assert _same(qn, want_q) and _same(kc, want_kc) and _same(vc, want_vc)


def test_what_is_out_of_range_is_recorded_and_not_written():
    B, T, page, lens = 4, 3, 16, [5, 14, 31, 2]
    q, k, v, wq, wk, c = _case(B, T, 4, 2, 64, page, lens, seed=5)
    good = _append(q, k, v, wq, wk, c)
    assert good[3] == bdla.OK
    width, n_pages = c["pages"].shape[1], c["kc"].shape[0]

    def changed(**kw):
        x = {n: t.clone() for n, t in c.items()}
        for name, (at, value) in kw.items():
            x[name][at] = value
        return x

    def rows_of(b, upto=T):
        """Cache rows that sequence b's first new tokens take."""
        pos = torch.arange(lens[b], lens[b] + upto, device="cuda")
        return c["pages"][b].long()[pos // page], pos % page

    # sequence 1 lies on two pages (14, 15 | 16)
    for x, lost in ((changed(pages=((1, 1), -1)), 1), (changed(pages=((1, 1), n_pages)), 1), (changed(pages=((1, 0), 2 ** 31 - 1)), 2),
                    (changed(lens=(1, -1)), 3), (changed(lens=(1, width * page)), 3), (changed(lens=(1, 2 ** 31 - 1)), 3),
                    (changed(lens=(1, 2 ** 31 - 4)), 3)):
        qn, kc, vc, status = _append(q, k, v, wq, wk, x)
        assert status == bdla.ERR_DEVICE
        want_k, want_v = good[1].clone(), good[2].clone()
        p, r = rows_of(1)
        drop = slice(0, 2) if lost == 2 else slice(2, 3) if lost == 1 else slice(0, 3)
        want_k[p[drop], r[drop]] = want_v[p[drop], r[drop]] = float("nan")
        assert _same(kc.isnan().to(BF16), want_k.isnan().to(BF16)) and torch.equal(kc.nan_to_num(), want_k.nan_to_num())
        assert torch.equal(vc.nan_to_num(), want_v.nan_to_num())
        keep = [0, 2, 3]
        assert _same(qn[keep], good[0][keep])
    for rows, counts, written in (([0, T, 1], T, (0, 2)), ([0, -1, 1], T, (0, 2)), (None, T + 1, (0, 1, 2)), (None, -1, ())):
        r = torch.tensor([[0, 1, 2]] * B, dtype=I32, device="cuda")
        n = torch.full((B,), T, dtype=I32, device="cuda")
        if rows is not None:
            r[2] = torch.tensor(rows, dtype=I32)
        n[2] = counts
        qn, kc, vc, status = _append(q, k, v, wq, wk, c, rows=r, counts=n)
        assert status == bdla.ERR_DEVICE
        p, at = rows_of(2)
        for j in range(T):
            assert bool(kc[p[j], at[j]].isnan().all()) == (j not in written) == bool(vc[p[j], at[j]].isnan().all())
        for b in (0, 1, 3):
            p, at = rows_of(b)
            assert _same(kc[p, at], good[1][p, at]) and _same(vc[p, at], good[2][p, at])
        assert _same(qn, good[0])


def test_malformed_offsets_are_recorded_and_stay_inside():
    lens = [3, 3, 3]
    q, k, v, wq, wk, c = _case(1, 20, 2, 1, 64, 16, lens, news=[20, 20, 20], seed=6)
    for cu in ([0, 8, 5, 20], [1, 8, 9, 20], [0, 8, 9, 19], [0, 30, 9, 20], [5, 4, 3, 2], [0, 8, 9, 40]):
        got = _append(q, k, v, wq, wk, c, cu_seqlens=torch.tensor(cu, dtype=I32, device="cuda"))
        assert got[3] == bdla.ERR_DEVICE, cu
    got = _append(q[:, :0], k[:, :0], v[:, :0], wq, wk, c, cu_seqlens=torch.tensor([0, 0, 0, 7], dtype=I32, device="cuda"))
    assert got[3] == bdla.ERR_DEVICE and got[0].shape == (1, 0, 2, 64)


def test_no_tokens_write_nothing():
    q, k, v, wq, wk, c = _case(2, 4, 2, 1, 64, 16, [3, 4], seed=7)
    qn, kc, vc, status = _append(q[:, :0], k[:, :0], v[:, :0], wq, wk, c)
    assert status == bdla.OK and qn.shape == (2, 0, 2, 64) and _same(kc, c["kc"]) and _same(vc, c["vc"])


def test_a_far_position_and_an_empty_table():
    """One token 2^31 - 20 positions into its context: the table's width alone makes that too far, which is recorded."""
    q, k, v, wq, wk, c = _case(1, 1, 4, 2, 128, 64, [0], seed=8)
    far = 2 ** 31 - 20
    c["lens"][0] = far
    qn, kc, _, status = _append(q, k, v, wq, wk, c)
    assert status == bdla.ERR_DEVICE and _same(kc, c["kc"])
    R = ref.rotation(torch.tensor([[far]], dtype=torch.float64, device="cuda"), 128, 10000.0, 128, False)
    ref.check("q", qn, ref.norm(q, wq, R, 1e-6))
    c["pages"], c["lens"][0] = c["pages"][:, :0], 0
    assert _append(q, k, v, wq, wk, c)[3] == bdla.ERR_DEVICE
    c["kc"] = c["vc"] = c["kc"][:0]
    assert _append(q, k, v, wq, wk, c)[3] == bdla.ERR_DEVICE


def test_what_is_not_finite_stays_in_its_head():
    q, k, v, wq, wk, c = _case(3, 5, 4, 2, 64, 16, [1, 2, 3], seed=9, views=False)
    good = _append(q, k, v, wq, wk, c)
    q[1, 2, 3, 7], k[2, 0, 1, 0], v[0, 4, 0, 63] = float("nan"), float("inf"), float("inf")
    bad = _append(q, k, v, wq, wk, c)
    differ = lambda x, y: ((x.view(torch.int16) != y.view(torch.int16)).reshape(-1, 64).any(1)).sum()
    assert int(differ(bad[0], good[0])) == 1 and int(differ(bad[1], good[1])) == 1
    assert int((bad[2].view(torch.int16) != good[2].view(torch.int16)).sum()) == 1


def test_another_stream_and_a_replayed_graph():
    q, k, v, wq, wk, c = _case(4, 1, 8, 2, 128, 16, [15, 0, 33, 7], seed=10)
    want = _append(q, k, v, wq, wk, c)
    side, ws = torch.cuda.Stream(), bdla.Workspace(256, "cuda")
    kc, vc = c["kc"].clone(), c["vc"].clone()
    torch.cuda.synchronize()
    qn = bdla.qk_norm_append(q, k, v, wq, wk, kc, vc, c["pages"], c["lens"], ws=ws, stream=side)
    side.synchronize()
    assert _same(qn, want[0]) and _same(kc, want[1]) and _same(vc, want[2])
    kc, vc = c["kc"].clone(), c["vc"].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qn = bdla.qk_norm_append(q, k, v, wq, wk, kc, vc, c["pages"], c["lens"], ws=ws)
    for step in range(3):   # the lengths move on between replays
        want_kc, want_vc = kc.clone(), vc.clone()
        graph.replay()
        want_q = bdla.qk_norm_append(q, k, v, wq, wk, want_kc, want_vc, c["pages"], c["lens"])
        assert _same(qn, want_q) and _same(kc, want_kc) and _same(vc, want_vc), step
        c["lens"] += 1
    assert ws.read_device_status() == bdla.OK
    c["lens"][1] = -5
    graph.replay()
    assert ws.read_device_status() == bdla.ERR_DEVICE


def test_arguments_are_refused_by_name(monkeypatch):
    q, k, v, wq, wk, c = _case(2, 3, 4, 2, 64, 16, [1, 2], seed=11)
    call = lambda **kw: bdla.qk_norm_append(kw.get("q", q), kw.get("k", k), kw.get("v", v), kw.get("wq", wq), kw.get("wk", wk),
                                            kw.get("kc", c["kc"]), kw.get("vc", c["vc"]), kw.get("pages", c["pages"]),
                                            kw.get("lens", c["lens"]), **{n: kw[n] for n in ("rows", "counts", "ws") if n in kw})
    call()
    for change, message in ((dict(k=k[:1]), "shapes disagree"), (dict(v=v[:, :2]), "v: batch rows"), (dict(v=v.float()), "v must be bf16"),
                            (dict(v=v.transpose(2, 3)), "v"), (dict(wq=wq.double()), "wq"), (dict(kc=c["kc"][:, :, :1].contiguous()), "cache must be"),
                            (dict(pages=c["pages"][:1]), "pages"), (dict(lens=c["lens"].long()), "lens"), (dict(v=v.cpu()), "v must be"),
                            (dict(rows=torch.zeros((2, 2), dtype=I32, device="cuda")), "rows"),
                            (dict(counts=torch.zeros(3, dtype=I32, device="cuda")), "counts"),
                            (dict(ws=bdla.Workspace(256, "cpu")), "ws is on cpu")):
        with pytest.raises(ValueError, match=message):
            call(**change)
    wide = torch.zeros((2, 3, 2, 68), dtype=BF16, device="cuda")
    with pytest.raises(bdla.BdlaError) as e:
        call(v=wide[..., :64])
    assert e.value.status == bdla.ERR_ALIGN
    monkeypatch.setattr(bdla, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        call()


def _held(c, kc):
    """Rows [sequence, position] of the cache as the tables order them."""
    return kc[c["pages"].long()].flatten(1, 2)


@pytest.mark.parametrize("cu,covered", [([1, 8, 9, 20], (1, 20)), ([0, 8, 9, 19], (0, 19)), ([0, 8, 9, 40], (0, 20)),
                                        ([20, 20, 20, 20], (20, 20)), ([-3, 2, 2, 9], (0, 9))])
def test_tokens_of_no_sequence_are_not_written(cu, covered):
    """Offsets in order that leave tokens out, or go past them: what is theirs is written, every other row stays as it was."""
    lens, T = [3, 0, 30], 20
    q, k, v, wq, wk, c = _case(1, T, 4, 2, 64, 16, lens, news=[T, T, T], seed=12)
    qn, kc, vc, status = _append(q, k, v, wq, wk, c, cu_seqlens=torch.tensor(cu, dtype=I32, device="cuda"))
    assert status == bdla.ERR_DEVICE
    want_k, want_v = c["kc"].clone(), c["vc"].clone()
    pos = torch.zeros((1, T), dtype=I32, device="cuda")
    at = {}
    for b, n in enumerate(lens):
        for t in range(max(cu[b], 0), min(cu[b + 1], T)):
            pos[0, t] = n + t - cu[b]
            at[t] = (c["pages"][b].long()[int(pos[0, t]) // 16], int(pos[0, t]) % 16)
    assert sorted(at) == list(range(*covered))
    all_q, all_k = bdla.qk_norm(q, k, wq, wk, positions=pos)
    for t, (page, row) in at.items():
        want_k[page, row], want_v[page, row] = all_k[0, t], v[0, t]
    assert _same(kc, want_k) and _same(vc, want_v)
    assert _same(qn[:, slice(*covered)], all_q[:, slice(*covered)]) and bool(qn.isfinite().all())


@pytest.mark.parametrize("cu", [[0, 8, 5, 20], [0, 30, 9, 20], [5, 4, 3, 2], [0, -9, 2 ** 31 - 1, 20], [2 ** 31 - 1, -(2 ** 31), 0, 20]])
def test_offsets_out_of_order_write_nothing_outside(cu):
    """Whatever they hold: pages that no table names and positions of the contexts stay as they were, and a row that is
    written is a token's, once."""
    lens, T = [3, 0, 30], 20
    q, k, v, wq, wk, c = _case(1, T, 4, 2, 64, 16, lens, news=[T, T, T], seed=13)
    qn, kc, vc, status = _append(q, k, v, wq, wk, c, cu_seqlens=torch.tensor(cu, dtype=I32, device="cuda"))
    assert status == bdla.ERR_DEVICE and bool(qn.isfinite().all())
    named = torch.zeros(kc.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, c["pages"].flatten().long(), True)
    assert not bool(named.all())
    tokens = []
    for new, old in ((kc, c["kc"]), (vc, c["vc"])):
        assert _same(new[~named], old[~named])
        held = _held(c, new)
        wrote = ~held.isnan().all(-1).all(-1)
        for b, n in enumerate(lens):
            assert not bool(wrote[b, :n].any())
        assert not bool(held[wrote].isnan().any()) and int(wrote.sum()) <= T
        tokens.append((held, wrote))
    assert torch.equal(tokens[0][1], tokens[1][1])
    is_token = (tokens[1][0][tokens[1][1]][:, None] == v[0][None]).flatten(2).all(2)   # [written, T]
    assert bool((is_token.sum(1) == 1).all()) and bool((is_token.sum(0) <= 1).all())
