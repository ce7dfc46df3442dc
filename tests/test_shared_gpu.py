"""Attention over shared pages against the definition in 64 bits over each sequence's own table, and the calls that it has to
refuse, record or survive."""
import pytest
import torch

import _attn_ref as ref
from chunked_linear_attention_bounded_gb300 import bdla

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(autouse=True)
def whatever_is_shared():
    """Small sizes too: by itself a call joins nothing that costs more than reading it again."""
    bdla.set_share_least(0)
    yield
    bdla.set_share_least(-1)


def _batch(groups, loose, own, T, Hq, Hk, d, page, seed=1, tree=False, spare=2, odd=0):
    """groups: (sequences, shared pages) each; then `loose` sequences; own: positions of each sequence behind what it
    shares.  Tables of a group begin with the same pages; what no table names, and what lies past a sequence's new tokens,
    is NaN.  `odd` positions of the last shared page are left out of what the call is told."""
    g = torch.Generator("cuda").manual_seed(seed)
    B = sum(n for n, _ in groups) + loose
    whole = [p for n, p in groups for _ in range(n)] + [0] * loose
    lens = [w * page + own[b % len(own)] for b, w in enumerate(whole)]
    need = [-(-(n + T) // page) for n in lens]
    total = sum(p for _, p in groups) + sum(e - w for e, w in zip(need, whole)) + spare
    order = torch.randperm(total, generator=g, device="cuda").to(I32)
    table = torch.full((B, max(need) + 1), -1, dtype=I32, device="cuda")
    at = b = 0
    cu = [0]
    for n, p in groups:
        table[b:b + n, :p] = order[at:at + p]
        at, b = at + p, b + n
        cu.append(b)
    kc, vc = (torch.randn((total, page, Hk, d), generator=g, device="cuda").to(BF16) for _ in "kv")
    for b in range(B):
        table[b, whole[b]:need[b]] = order[at:at + need[b] - whole[b]]
        at += need[b] - whole[b]
        if (lens[b] + T) % page:
            last = int(table[b, need[b] - 1])
            kc[last, (lens[b] + T) % page:] = vc[last, (lens[b] + T) % page:] = float("nan")
    kc[order[at:].long()] = vc[order[at:].long()] = float("nan")
    q = (torch.randn((B, T, Hq, d), generator=g, device="cuda") * 1.5).to(BF16)
    masks = None
    if tree:
        masks = torch.zeros((B, T), dtype=torch.int64)
        bits = torch.rand((B, T, T), generator=torch.Generator().manual_seed(seed)) < 0.4
        for i in range(T):
            for j in range(i):
                masks[:, i] |= bits[:, i, j].long() << j
            masks[:, i] |= (1 << i) if i < 63 else -(1 << 63)
        if T > 2:
            masks[:, T // 2] = 0
        masks = masks.cuda()
    i32 = lambda x: torch.tensor(x, dtype=I32, device="cuda")
    return dict(q=q, kc=kc, vc=vc, table=table, lens=i32(lens), cu=i32(cu),
                shared=i32([max(p * page - odd, 0) for _, p in groups]), tree=masks)


def _call(x, ws=None, **kw):
    return bdla.attn_shared(x["q"], x["kc"], x["vc"], x["table"], x["lens"], x["cu"], x["shared"], tree=x["tree"], ws=ws, **kw)


def _holds(x, ws=None, status=bdla.OK):
    ws = ws or bdla.Workspace(256, "cuda")
    o, lse = _call(x, ws)
    tree = None if x["tree"] is None else x["tree"].cpu()
    want_o, want_l = ref.cached(x["q"], x["kc"], x["vc"], x["table"], x["lens"].tolist(), tree, x["q"].shape[3] ** -0.5)
    assert ws.read_device_status() == status
    ref.check("o", o, want_o)
    ref.check("lse", lse, want_l)
    return o, lse


CASES = {  # groups, loose, own, T, Hq, Hk, d, page, tree
    "one": ([(1, 5)], 0, [3], 1, 4, 2, 64, 16, False),
    "two rows": ([(2, 9)], 0, [0, 5], 1, 1, 1, 64, 16, False),
    "16 rows": ([(4, 40)], 0, [7, 0, 300, 41], 1, 8, 2, 128, 16, False),
    "32 rows": ([(4, 11)], 2, [7, 0, 300, 41], 2, 4, 1, 128, 48, False),
    "wide and narrow": ([(12, 33)], 0, [5, 0, 700, 64, 63], 1, 16, 4, 128, 16, False),
    "pages of one": ([(40, 190)], 1, [5, 0, 70], 1, 2, 2, 64, 1, False),
    "pages of 24": ([(9, 30)], 1, [5, 0, 70], 1, 8, 2, 128, 24, False),
    "pages of 256": ([(30, 3)], 1, [5, 0, 270], 1, 4, 2, 64, 256, False),
    "blocks of rows": ([(70, 20)], 0, [1, 40], 1, 8, 1, 128, 32, False),
    "many blocks": ([(150, 9)], 3, [1, 40, 9], 1, 16, 2, 64, 64, False),
    "groups of all kinds": ([(1, 30), (0, 4), (2, 30), (11, 0), (13, 17), (3, 2), (20, 40)], 5, [0, 9, 200, 33], 1, 12, 4, 64, 16, False),
    "several tokens": ([(6, 20), (5, 7)], 2, [0, 9, 130], 5, 8, 4, 128, 16, False),
    "rows of 32": ([(3, 20), (1, 4)], 2, [0, 9, 130], 8, 8, 2, 128, 16, True),
    "rows of 24": ([(3, 20), (5, 14)], 2, [0, 9, 530], 3, 8, 1, 64, 32, False),
    "64 rows in a short table": ([(16, 200)], 0, [0, 9, 130], 1, 8, 2, 128, 16, False),
    "64 rows in a long table": ([(16, 300)], 0, [0, 9, 130], 1, 8, 2, 128, 16, False),
    "trees": ([(5, 20), (2, 7)], 2, [0, 9, 130], 17, 8, 4, 64, 48, True),
    "wide trees": ([(3, 20), (4, 7), (1, 5)], 2, [0, 9, 130, 400], 21, 8, 2, 128, 16, True),
    "trees of 64": ([(2, 12)], 1, [0, 190], 64, 8, 1, 64, 100, True),
    "trees past 256 rows": ([(2, 12), (2, 3)], 1, [0, 190], 40, 16, 2, 128, 64, True),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("odd,least", [(0, 0), (7, 0), (0, -1)])
def test_the_definition(name, odd, least):
    bdla.set_share_least(least)
    groups, loose, own, T, Hq, Hk, d, page, tree = CASES[name]
    _holds(_batch(groups, loose, own, T, Hq, Hk, d, page, seed=len(name), tree=tree, odd=odd))


def test_what_the_call_is_told_is_a_hint():
    """Nothing, a part, all, and more than all members have: the same attention.  In the last case the sequences' common
    pages go on behind the shortest context."""
    x = _batch([(7, 30), (4, 12)], 1, [0, 17, 160], 2, 8, 2, 64, 16)
    for told in ([0, 0], [64, 63], [479, 1], [480, 192], [10 ** 9, 2 ** 31 - 1]):
        x["shared"] = torch.tensor(told, dtype=I32, device="cuda")
        if max(told) > 480:
            x["lens"] = torch.tensor([480, 470, 455, 478, 300, 64, 100] + [192, 150, 100, 130] + [17], dtype=I32, device="cuda")
        _holds(x)


def test_a_sequence_with_nothing_to_see():
    x = _batch([(3, 0), (2, 9)], 1, [0], 2, 16, 4, 64, 16)
    x["tree"] = torch.zeros((6, 2), dtype=torch.int64, device="cuda")
    o, lse = _holds(x)
    assert not bool(o[[0, 1, 2, 5]].any()) and bool((lse[[0, 1, 2, 5]] == -float("inf")).all())
    x = _batch([(40, 0)], 0, [0], 20, 8, 2, 128, 16)   # rows of the wide kernel without a single tile
    x["lens"][7] = -4
    x["tree"] = torch.zeros((40, 20), dtype=torch.int64, device="cuda")
    o, lse = _holds(x, status=bdla.ERR_DEVICE)
    assert not bool(o.any()) and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("many", [False, True])
def test_bad_pages_are_recorded_and_not_seen(many):
    x = _batch([(12 if many else 3, 30), (2, 10)], 1, [40, 5], 1, 8, 2, 128, 16)
    n = x["table"].shape[0] - 3   # sequences of the first group
    _holds(x)
    for at, value in ((4, -1), (29, x["kc"].shape[0]), (0, 2 ** 31 - 1)):
        y = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
        y["table"][:n, at] = value
        _holds(y, status=bdla.ERR_DEVICE)
    y["table"], y["lens"] = x["table"].clone(), x["lens"].clone()
    y["table"][1, 30] = -5   # a page of one sequence's own
    _holds(y, status=bdla.ERR_DEVICE)


def test_only_the_first_sequences_table_is_read_for_what_is_shared():
    x = _batch([(9, 30)], 0, [40, 5], 1, 8, 2, 128, 16)
    want = _holds(x)
    x["table"][1:, :30] = -1
    got = _call(x)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_bad_offsets_and_lengths_are_recorded():
    x = _batch([(7, 30), (4, 12)], 1, [0, 17, 160], 1, 8, 2, 64, 16)
    good = x["cu"]
    for cu in ([0, 8, 7], [-1, 7, 11], [0, 7, 13], [5, 3, 11], [0, 7, 2 ** 31 - 1], [0, -(2 ** 31), 11]):
        x["cu"] = torch.tensor(cu, dtype=I32, device="cuda")
        _holds(x, status=bdla.ERR_DEVICE)   # every sequence by itself
    x["cu"] = torch.tensor([2, 2, 5], dtype=I32, device="cuda")   # in order: an empty group, part of the other
    x["shared"] = torch.tensor([480, 480], dtype=I32, device="cuda")
    _holds(x)
    x["cu"], x["shared"] = good, torch.tensor([480, -1], dtype=I32, device="cuda")
    _holds(x, status=bdla.ERR_DEVICE)
    x["shared"] = torch.tensor([480, 192], dtype=I32, device="cuda")
    keep = x["lens"].clone()
    for value in (-1, -(2 ** 31), x["table"].shape[1] * 16):
        x["lens"] = keep.clone()
        x["lens"][9] = value
        x["table"][9, 12:] = x["table"][8, 11]   # the positions up to the table's end exist
        _holds(x, status=bdla.ERR_DEVICE)
    x["lens"][9] = 2 ** 31 - 1
    _holds_far = bdla.Workspace(256, "cuda")
    _call(x, _holds_far)
    assert _holds_far.read_device_status() == bdla.ERR_DEVICE


def test_what_is_not_finite_stays_in_its_group():
    x = _batch([(12, 20), (3, 20)], 2, [40, 5], 1, 8, 2, 64, 16)
    want = _call(x)
    x["vc"][int(x["table"][0, 3]), 5, 1, 9] = float("inf")
    x["kc"][int(x["table"][13, 20]), 2, 0, 9] = float("nan")   # sequence 13's own
    o, lse = _call(x)
    keep = [12, 14, 15, 16]
    assert torch.equal(o[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])
    assert torch.equal(lse[:12], want[1][:12]) and torch.equal(o[:12, :, :4], want[0][:12, :, :4])
    assert not bool(o[:12, :, 4:, 9].isfinite().any())
    assert bool(o[13, :, :4].isnan().all()) and torch.equal(o[13, :, 4:], want[0][13, :, 4:])


def test_the_same_inputs_give_the_same_bits_and_other_streams_do_too():
    x = _batch([(30, 40), (3, 20)], 2, [40, 5, 700], 1, 8, 2, 128, 16)
    want = _holds(x)
    side, ws = torch.cuda.Stream(), bdla.Workspace(1 << 26, "cuda")
    torch.cuda.synchronize()
    for stream in (None, side, side):
        got = _call(x, ws, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    other = bdla.Workspace(1 << 26, "cuda")   # two calls at once, a workspace each
    torch.cuda.synchronize()
    got = [_call(x, w, stream=s) for _ in range(10) for w, s in ((ws, side), (other, None))]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for y in got for a, b in zip(y, want))


@pytest.mark.parametrize("T", [1, 12])
def test_a_replayed_graph_follows_lengths_groups_and_tables(T):
    x = _batch([(20, 25), (6, 9)], 3, [40, 5, 300], T, 8, 2, 128, 16)
    ws = bdla.Workspace(1 << 27, "cuda")
    _call(x, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = _call(x, ws)
    first = {k: v.clone() for k, v in x.items() if v is not None}
    for cu, shared, fewer in (([0, 20, 26], [400, 144], 0), ([0, 10, 26], [390, 0], 3), ([3, 3, 8], [100, 64], 40), ([0, 0, 0], [1, 1], 0)):
        x["cu"].copy_(torch.tensor(cu, dtype=I32))
        x["shared"].copy_(torch.tensor(shared, dtype=I32))
        x["lens"].copy_(torch.maximum(first["lens"] - fewer, torch.zeros_like(first["lens"])))
        o.zero_(), lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert ws.read_device_status() == bdla.OK
        want_o, want_l = ref.cached(x["q"], x["kc"], x["vc"], x["table"], x["lens"].tolist(), None, 128 ** -0.5)
        ref.check("o", o, want_o)
        ref.check("lse", lse, want_l)


def test_nothing_to_look_at():
    """Tables and caches without pages."""
    q, i32 = torch.randn((3, 1, 4, 64), device="cuda").to(BF16), lambda *v: torch.tensor(v, dtype=I32, device="cuda")
    kc, none = torch.zeros((0, 16, 2, 64), dtype=BF16, device="cuda"), torch.zeros((3, 0), dtype=I32, device="cuda")
    for table in (none, torch.zeros((3, 2), dtype=I32, device="cuda")):
        ws = bdla.Workspace(256, "cuda")
        o, lse = bdla.attn_shared(q, kc, kc, table, i32(0, 5, 9), i32(0, 3), i32(9), ws=ws)
        assert ws.read_device_status() == bdla.ERR_DEVICE
        assert not bool(o.any()) and bool((lse == -float("inf")).all())


def _off(got, want):
    return float((got.double() - want.double()).norm() / want.double().norm())


def test_long_and_many_against_attention_of_each_sequence():
    """Sizes too large for the definition row by row: both kernels are held to it elsewhere, and round o and the weights
    to bf16 on their own: each at most 2^-8 sqrt(2) of the norm off, and in practice half of it."""
    for groups, loose, own, T, Hq, Hk, d, page in (
            ([(24, 60001 // 64)], 0, [3, 900, 17], 1, 32, 8, 128, 64), ([(300, 40)], 7, [9, 0, 60], 1, 8, 8, 128, 16),
            ([(2, 3000)], 0, [9, 0], 1, 2, 1, 64, 16), ([(3, 9)] * 2800, 100, [1, 5, 2], 1, 2, 1, 64, 8)):
        x = _batch(groups, loose, own, T, Hq, Hk, d, page)
        ws = bdla.Workspace(256, "cuda")
        o, lse = _call(x, ws)
        want_o, want_l = bdla.attn_cached(x["q"], x["kc"], x["vc"], x["table"], x["lens"], ws=ws)
        assert ws.read_device_status() == bdla.OK
        assert _off(o, want_o) <= 2 * 2.0 ** -8 * 2 ** 0.5 and _off(lse, want_l) <= 2.0 ** -18
        del x


def test_a_cache_past_32_bit_offsets():
    """4.4e9 elements of keys, of which the sequences use the last pages."""
    Hk, d, page, n_pages = 8, 128, 64, 67600
    g = torch.Generator("cuda").manual_seed(3)
    kc, vc = (torch.empty((n_pages, page, Hk, d), dtype=BF16, device="cuda") for _ in "kv")
    for x in (kc, vc):
        x[-40:] = torch.randn((40, page, Hk, d), generator=g, device="cuda").to(BF16)
    table = torch.arange(n_pages - 40, n_pages, dtype=I32, device="cuda").view(1, 40).repeat(12, 1)
    q = torch.randn((12, 1, 16, d), generator=g, device="cuda").to(BF16)
    lens = torch.tensor([40 * page - 1 - 3 * b for b in range(12)], dtype=I32, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=I32, device="cuda")
    o, lse = bdla.attn_shared(q, kc, vc, table, lens, i32(0, 12), i32(2000))
    small = lambda c: c[-40:].clone()
    want_o, want_l = ref.cached(q, small(kc), small(vc), table - (n_pages - 40), lens.tolist(), None, d ** -0.5)
    ref.check("o", o, want_o)
    ref.check("lse", lse, want_l)


@pytest.mark.parametrize("role", [bdla.STALL_PRODUCER, bdla.STALL_MMA, bdla.STALL_EPILOGUE])
@pytest.mark.parametrize("page", [32, 24])   # by TMA, and row by row
def test_expired_waits(role, page):
    x = _batch([(30, 30)], 1, [9, 200], 1, 8, 2, 64, page)
    ws = bdla.Workspace(1 << 26, "cuda")
    try:
        bdla.set_wait_limit_ns(20_000_000)
        bdla.set_test_stall(bdla.KERNEL_ATTN_SHARED, role)
        _call(x, ws)
        assert ws.read_device_status() == bdla.ERR_TIMEOUT
    finally:
        bdla.set_test_stall(bdla.KERNEL_ATTN_SHARED, bdla.STALL_NONE)
        bdla.set_wait_limit_ns(0)
    _holds(x, ws)


def test_arguments_are_refused_by_name(monkeypatch):
    x = _batch([(3, 4)], 0, [1], 1, 4, 2, 64, 16)
    for change, message in ((dict(shared=x["shared"].long()), "shared"), (dict(shared=x["shared"][None]), "shared"),
                            (dict(cu=x["cu"][:1]), "cu_groups"), (dict(cu=x["cu"].float()), "cu_groups"), (dict(cu=x["cu"].cpu()), "cu_groups"),
                            (dict(table=x["table"][:1]), "pages"), (dict(lens=x["lens"][:1]), "lens"), (dict(q=x["q"].float()), "q must be"),
                            (dict(tree=torch.zeros((3, 2), dtype=torch.int64, device="cuda")), "tree"),
                            (dict(kc=x["kc"][..., :32].contiguous(), vc=x["vc"][..., :32].contiguous()), "widths")):
        with pytest.raises(ValueError, match=message):
            _call({**x, **change})
    none = dict(cu=torch.zeros(1, dtype=I32, device="cuda"), shared=torch.zeros(0, dtype=I32, device="cuda"))
    for change, status in ((none, bdla.ERR_SHAPE), (dict(q=x["q"][:, :0]), bdla.ERR_SHAPE), (dict(q=x["q"].repeat(1, 65, 1, 1)), bdla.ERR_UNSUPPORTED)):
        with pytest.raises(bdla.BdlaError) as e:
            _call({**x, **change})
        assert e.value.status == status
    with pytest.raises(ValueError, match="ws is on cpu"):
        _call(x, bdla.Workspace(256, "cpu"))
    monkeypatch.setattr(bdla, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        _call(x)
