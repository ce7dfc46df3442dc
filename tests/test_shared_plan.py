"""The plan of attention over shared pages, restated: that every row meets every position that it has to meet exactly once,
that the join finds the sums where the pieces put them, and that lists and partial sums stay inside what the sizes alone
give them."""
import random

import pytest

SMS, TILE, WIDE, NARROW = 152, 128, 256, 32
RUN = 10   # what a change of rows costs, in tiles of 128 rows
LEAST_WIDE, LEAST_NARROW, SHORT_TABLE, LEAST_LINE, N_SIZES = 32_000_000, 2_000_000, 4096, 2 + RUN, 8


def up(a, b):
    return -(-a // b)


class Sizes:
    def __init__(s, B, T, G, Hk, d, n_groups, max_keys):
        s.B, s.T, s.G, s.Hk, s.d, s.n_groups = B, T, G, Hk, d, n_groups
        R, every = T * G, T * G * B
        s.own_wide = R > NARROW
        s.wide = s.own_wide or every > (NARROW if max_keys > SHORT_TABLE else 2 * NARROW)
        s.mr = 16 if R <= 16 else 32
        s.slots = SMS * ((9 if d == 128 else 16) if s.mr == 16 else 3 if d == 128 else 4)
        s.extra = 2 * up(s.slots, Hk)
        s.most = 0 if s.own_wide else B + 2 * min(n_groups, B // 2) + 4 + s.extra
        s.rows = 0
        if s.wide:
            s.rows += 2 * every * Hk * (2 if s.own_wide else 1) + WIDE * SMS
        if not s.own_wide:
            s.rows += (2 * every + NARROW * s.extra) * Hk


def plan(z, cu, shared, lens, cap, thrift=1):
    NG, E = z.n_groups, z.n_groups + z.B
    n = [min(max(x, 0), cap) for x in shared]
    bad = any(cu[g] < 0 or cu[g + 1] < cu[g] or cu[g + 1] > z.B for g in range(NG))
    group = [-1] * z.B
    for b in range(z.B):
        if not bad:
            lo, hi = 0, NG
            while lo < hi:
                mid = (lo + hi + 1) // 2
                lo, hi = (mid, hi) if cu[mid] <= b else (lo, mid - 1)
            group[b] = lo if lo < NG and cu[lo] <= b else -1
        if group[b] >= 0:
            n[group[b]] = min(n[group[b]], max(lens[b], 0))
    for g in range(NG):
        m = 0 if bad else cu[g + 1] - cu[g]
        least = LEAST_WIDE if z.wide and not z.own_wide and m * z.T * z.G > NARROW else LEAST_NARROW
        if m < 2 or (m - 1) * n[g] * z.Hk * z.d * 2 < least * thrift:
            n[g] = 0
    for b in range(z.B):
        end = 0 if lens[b] < 0 else min(lens[b] + z.T, cap)
        n.append(end - (n[group[b]] if group[b] >= 0 else 0))

    def entry(e):
        R, tok0, wide = z.T * z.G, (e - NG) * z.T, z.own_wide
        if e < NG:
            tok0, R = (cu[e] * z.T, (cu[e + 1] - cu[e]) * z.T * z.G) if n[e] > 0 else (0, 0)
            wide = z.wide and R > NARROW
        return R, tok0, wide, up(R, z.mr)

    entries = [entry(e) for e in range(E)]
    full, single = lambda R: up(R, TILE) // 2, lambda R: up(R, TILE) % 2   # blocks of two row tiles, and of one
    line_of = lambda R, nt: z.Hk * (full(R) * (2 * nt + RUN) + single(R) * (nt + RUN)) if nt else 0
    tiles = sum(line_of(x[0], up(n[e], TILE)) for e, x in enumerate(entries) if x[2])
    positions = sum(x[3] * n[e] for e, x in enumerate(entries) if not x[2])
    per_cta = max(LEAST_LINE, up(tiles, SMS))
    size = min(up(up(positions, z.extra), 64) * 64, 2 ** 31 - 128) if z.most > 0 else 64
    if z.most > 0 and size <= 128 << (N_SIZES - 1):
        best = None
        for s in (128 << i for i in range(N_SIZES)):
            pieces = sum(x[3] * max(up(n[e], s), 1 if e >= NG else 0) for e, x in enumerate(entries) if not x[2])
            longest = max([up(n[e], s) for e, x in enumerate(entries) if not x[2]], default=0)
            cost = (positions + 128 * pieces) * z.Hk / z.slots + s + 4 * longest
            if s >= size and (best is None or cost < best[0]):
                best = (cost, s)
        size = best[1]
    parts, wides, work, base, rows, first_entry = [], [], [], 0, 0, {}
    for e, (R, tok0, wide, blocks) in enumerate(entries):
        g = group[e - NG] if e >= NG else -1
        first = 0 if e < NG or g < 0 else n[g]
        b = e - NG if e >= NG else (cu[e] if n[e] > 0 else 0)
        np, direct, nt = 0, False, up(n[e], TILE) if wide else 0
        w = line_of(R, nt)
        need = (up(2 * nt if full(R) else nt, per_cta) + 1) * R * z.Hk if nt else 0
        if not wide:
            np = up(n[e], size)
            if e >= NG:
                np = max(np, 1)
                direct = np == 1 and (g < 0 or n[g] == 0)
            need = 0 if direct else np * R * z.Hk
        base1 = base + z.Hk * full(R) * (2 * nt + RUN)
        parts.append((base, nt, R, rows, -1 if direct else np, tok0, base1, full(R)))
        if nt:
            for start, end, rb0, rb1, rt in ((base, base1, 0, full(R), 2), (base1, base + w, full(R), full(R) + 1, 1)):
                if start == end:
                    continue
                for c in range(up(start, per_cta), up(end, per_cta)):
                    first_entry[c] = len(wides)
                wides.append((start, b, tok0, R, first, first + n[e], nt, rows, rb0, rb1, rt))
        for i in range(np):
            for rb in range(blocks):
                work.append((b, first + min(n[e], i * size), first + min(n[e], (i + 1) * size), tok0, R, rb * z.mr,
                             -1 if direct else rows + i * z.Hk * R))
        base, rows = base + w, rows + need
    assert base == tiles
    return group, parts, wides, work, rows, tiles, per_cta, first_entry


def walk(z, wides, tiles, per_cta, first_entry, cta):
    """(entry, block of rows, key head, first tile, tiles, piece) of each run of a CTA of the wide kernel."""
    x = cta * per_cta
    end = min(tiles, x + per_cta)
    if x >= tiles:
        return
    e = first_entry[cta]
    base, nt, rt = wides[e][0], wides[e][6], wides[e][10]
    unit = (x - base) // (nt * rt + RUN)
    start = base + unit * (nt * rt + RUN) + RUN
    t0, rb, kh, piece = max(up(x - start, rt), 0), unit // z.Hk + wides[e][8], unit % z.Hk, cta - start // per_cta
    while True:
        nt, rt = wides[e][6], wides[e][10]
        at = start + t0 * rt
        n = min(nt - t0, up(end - at, rt)) if at < end else 0
        if n > 0:
            yield e, rb, kh, t0, n, piece
        start += nt * rt + RUN
        t0 = piece = 0
        if start >= end:
            return
        kh += 1
        if kh == z.Hk:
            kh, rb = 0, rb + 1
            if rb == wides[e][9]:
                e += 1
                rb = wides[e][8]


def check(B, T, G, Hk, d, cu, shared, lens, cap, thrift=0):
    z = Sizes(B, T, G, Hk, d, len(shared), cap)
    group, parts, wides, work, rows, tiles, per_cta, first_entry = plan(z, cu, shared, lens, cap, thrift)
    assert rows <= z.rows and len(work) <= z.most and tiles <= SMS * per_cta and all(0 <= c < SMS for c in first_entry)
    # what each piece leaves, by its row of the partial sums: (token, query head) and positions
    left, done = {}, {}

    def put(at, token, head, a, e):
        if at is None:
            assert (token, head) not in done
            done[token, head] = [(a, e)]
        else:
            assert 0 <= at < z.rows and at not in left, at
            left[at] = (token, head, a, e)

    for b, a, e, tok0, R, row0, part in work:
        for kh in range(Hk):
            for r in range(row0, min(R, row0 + z.mr)):
                put(None if part < 0 else part + kh * R + r, tok0 + r // G, kh * G + r % G, a, e)
    for cta in range(SMS):
        for i, rb, kh, t0, n, piece in walk(z, wides, tiles, per_cta, first_entry, cta):
            base, b, tok0, R, first, end, nt, part, rb0, rb1, rt = wides[i]
            assert rb0 <= rb < rb1 and up(min(R, rb * WIDE + WIDE) - rb * WIDE, TILE) == rt
            for r in range(rb * WIDE, min(R, rb * WIDE + WIDE)):
                put(part + (piece * Hk + kh) * R + r, tok0 + r // G, kh * G + r % G, first + t0 * TILE,
                    min(end, first + (t0 + n) * TILE))

    def pieces(e, b, i, h):
        base, nt, R, part, np, tok0, base1, full = parts[e]
        rr, kh = (b * T + i - tok0) * G + h % G, h // G
        if nt:
            rb, rt = rr // WIDE, 2 if rr // WIDE < full else 1
            begin = RUN + (base + (rb * Hk + kh) * (2 * nt + RUN) if rb < full else base1 + kh * (nt + RUN))
            np = (begin + (nt - 1) * rt) // per_cta - begin // per_cta + 1
        return [part + kh * R + rr + s * Hk * R for s in range(max(np, 0))] if np >= 0 else None

    used = set()
    for b in range(B):
        end = 0 if lens[b] < 0 else min(lens[b] + T, cap)
        for i in range(T):
            for h in range(G * Hk):
                own = pieces(z.n_groups + b, b, i, h)
                if own is None:
                    spans = done[b * T + i, h]
                else:
                    at = (pieces(group[b], b, i, h) if group[b] >= 0 else []) + own
                    used.update(at)
                    assert all(left[x][:2] == (b * T + i, h) for x in at)
                    spans = [left[x][2:] for x in at]
                spans = [s for s in spans if s[0] < s[1]]
                assert (spans[0][0] if spans else 0) == 0 and (spans[-1][1] if spans else 0) == end
                assert all(x[1] == y[0] for x, y in zip(spans, spans[1:]))
    assert used == set(left)   # nothing is summed that nobody joins


def test_small_and_odd():
    check(1, 1, 1, 1, 64, [0, 1], [100], [200], 1024)
    check(2, 1, 1, 1, 64, [0, 2], [100], [200, 64], 1024)
    check(2, 1, 4, 2, 128, [0, 2], [0], [0, 0], 0)
    check(3, 2, 4, 2, 128, [0, 2], [500], [-1, 700, 9], 640)          # a bad length, one past the table
    check(9, 5, 8, 1, 64, [0, 9], [4000], [4000] * 9, 8192)
    check(4, 64, 8, 1, 128, [1, 3], [900], [900, 1000, 901, 5], 2048)  # trees of several blocks of rows
    check(3, 1, 2, 2, 64, [2, 1], [5], [100, 100, 100], 1024)          # malformed: nobody shares


# thrift 0: whatever is shared counts, so that small sizes show how it is cut
@pytest.mark.parametrize("thrift", [0, 1])
@pytest.mark.parametrize("seed", range(60))
def test_every_position_once(seed, thrift):
    r = random.Random(seed)
    B = r.choice([1, 2, 3, 8, 17, 40])
    T, G, Hk = r.choice([1, 1, 2, 7, 20]), r.choice([1, 2, 4, 8]), r.choice([1, 2, 3, 8])
    NG = r.randint(1, min(B, 5))
    cu = sorted(r.randint(0, B) for _ in range(NG + 1))
    top = r.choice([50, 1000, 20000])
    lens = [r.randint(0, top) for _ in range(B)]
    shared = [r.choice([0, 63, 64, r.randint(0, top), 10 ** 9]) for _ in range(NG)]
    if r.random() < 0.6:   # contexts that are longer than what is shared
        lens = [n + max(min(shared[g], top) for g in range(NG)) for n in lens]
    check(B, T, G, Hk, r.choice([64, 128]), cu, shared, lens, max(lens) + r.choice([T, T + 77, 1]),
          thrift)


def test_bounds_at_large_sizes():
    """Lists and partial sums of batches too large to follow row by row."""
    r = random.Random(1)
    for B, T, G, Hk, NG, top in ((256, 1, 4, 8, 1, 131072), (256, 1, 4, 8, 128, 131072), (256, 1, 1, 1, 100, 1 << 21),
                                 (600, 8, 4, 8, 3, 1 << 17), (5000, 1, 8, 1, 2500, 40000), (64, 64, 8, 8, 9, 1 << 16)):
        z = Sizes(B, T, G, Hk, 128, NG, 1 << 30)
        cu = [B * g // NG for g in range(NG + 1)]
        for kind in range(3):
            shared = [r.randint(top // 2, top) if kind else top for _ in range(NG)]
            lens = [top + (r.randint(0, top) if kind == 2 else 5) for _ in range(B)]
            _, _, _, work, rows, tiles, per_cta, first = plan(z, cu, shared, lens, 1 << 30, kind % 2)
            assert rows <= z.rows and len(work) <= z.most and tiles <= SMS * per_cta and all(c < SMS for c in first)


def _bytes(z):
    """The workspace: the status word, then each table of the plan on its own lines of 256 bytes."""
    entries = z.n_groups + z.B
    ints = 3 * z.n_groups + 2 * z.B + 1
    sizes = (24, 2 * entries * 48, entries * 32, z.most * 32, SMS * 4, z.B * 4, ints * 4, z.rows * z.d * 4, z.rows * 8)
    return 256 + sum(up(n, 256) * 256 for n in sizes)


def test_the_library_asks_for_what_is_restated_here():
    """Rows of partial sums, the list's length and the tables' sizes, by the bytes of workspace that they come to."""
    from chunked_linear_attention_bounded_gb300 import bdla
    from chunked_linear_attention_bounded_gb300.build import build
    build()
    r = random.Random(7)
    for _ in range(400):
        B, T = r.choice([1, 2, 7, 60, 256, 1000]), r.choice([1, 1, 2, 5, 17, 64])
        G, Hk, d = r.choice([1, 2, 4, 8]), r.choice([1, 2, 4, 8]), r.choice([64, 128])
        n_groups, keys = r.randint(1, min(2 * B, 300)), r.choice([0, 64, 4096, 4097, 1 << 17])
        got = bdla.lib().bdla_workspace_bytes_attn(bdla.ATTN_SHARED, bdla.AttnDims(B, T, G * Hk, Hk, d), n_groups, keys)
        z = Sizes(B, T, G, Hk, d, n_groups, keys)
        assert got == (_bytes(z) if z.rows < 1 << 31 else 0), (B, T, G, Hk, d, n_groups, keys)
