"""How a latent tree call is shared out, restated from the kernels' header
(latent_work.cuh) and entry point: which kernel takes it, in how many parts,
which tiles of which unit a part computes, what is left to the join.

A unit is (sequence, 128 or 16 query rows): its tree tiles, then its prefix
tiles.  It weighs its tiles and a fixed weight in front of them; a sequence whose
length is refused (None here) has units without tiles."""
from dataclasses import dataclass, field

PAIRS = dict(tile=128, rows=128, fixed=3, join=6, most=76)
FEW = dict(tile=64, rows=16, fixed=2, join=4, most=152)


def up(a, b):
    return -(-a // b)


def takes_few(batch, nodes, heads, latent, max_prefix):
    rows, units = nodes * heads, batch * up(nodes * heads, 16)
    tiles = units * (up(max_prefix, 64) + up(nodes, 64))
    return rows <= 16 or (units <= 152 and tiles <= (1064 if latent == 512 else 456))


def n_parts(k, batch, nodes, heads, max_prefix):
    tiles = batch * up(nodes * heads, k["rows"]) * (up(max_prefix, k["tile"]) + up(nodes, k["tile"]))
    return min(tiles if k is FEW else (tiles + 1) // 2, k["most"])


@dataclass
class Plan:
    kernel: str
    form: int                                     # of the join
    mode: str                                     # "whole", "cut" or "halves"
    parts: int
    used: int                                     # parts that have a range
    segments: list = field(default_factory=list)  # of each part: (sequence, unit, t0, t1, T)
    cuts: dict = field(default_factory=dict)      # part -> (sequence, unit, parts): what the join adds up, as the kernel finds it


def plan(lengths, nodes, heads, latent, max_prefix=None):
    batch = len(lengths)
    max_prefix = max(x or 0 for x in lengths) if max_prefix is None else max_prefix
    few = takes_few(batch, nodes, heads, latent, max_prefix)
    k = FEW if few else PAIRS
    parts, fixed, rows_all = n_parts(k, batch, nodes, heads, max_prefix), k["fixed"], nodes * heads
    rt = up(rows_all, k["rows"])
    tiles = [0 if x is None else up(nodes, k["tile"]) + up(x, k["tile"]) for x in lengths]
    total, most, units = sum(rt * (t + fixed) for t in tiles), max(tiles) + fixed, batch * rt
    first = [0]
    for t in tiles:
        first.append(first[-1] + rt * (t + fixed))
    cut = min(units, parts - 1)
    rows = min(rows_all, k["rows"]) * cut
    p = Plan("few" if few else "pairs", 8 if rows <= 256 else 1 if few or rows <= 4096 else 0, "cut", parts, parts)

    each = 1 if units <= parts else up(units, parts)
    if 5 * each * most * parts <= 6 * total + 5 * k["join"] * parts:
        p.mode = "whole"
        start = lambda u: first[u // rt] + (u % rt) * (tiles[u // rt] + fixed) if u < units else total  # noqa: E731
        ranges = [(start(each * i), start(each * (i + 1))) if each * i < units else (0, 0) for i in range(parts)]
    else:
        n = min(total, parts)
        far = (100 << 20) // (k["tile"] * (latent + 64) * 2)
        if rt > 1 and units * most == total and most * batch > far:
            even = 2 * parts // units * units // 2
            if 10 * even >= 9 * parts and even < n:
                n, p.mode = even, "halves"
        ranges = [(total * i // n, total * (i + 1) // n) if i < n else (0, 0) for i in range(parts)]
        for i in range(1, n):        # as the part that begins inside a unit finds it
            lo, before = ranges[i][0], ranges[i - 1][0]
            b = max(x for x in range(batch) if first[x] <= lo)
            unit = (lo - first[b]) // (tiles[b] + fixed)
            begin = first[b] + unit * (tiles[b] + fixed) + fixed
            if tiles[b] > 0 and lo > begin and before <= begin:
                e = up((begin + tiles[b]) * n, total) - 1
                p.cuts[i] = (b, unit, min(e, n - 1) - i + 2)
    p.used = sum(hi > lo for lo, hi in ranges)
    for lo, hi in ranges:
        mine = []
        for b in range(batch):
            w = tiles[b] + fixed
            if not tiles[b] or hi <= first[b] or lo >= first[b + 1]:
                continue
            for u in range(max(0, (lo - first[b]) // w), min(rt, up(hi - first[b], w))):
                begin = first[b] + u * w + fixed
                t0, t1 = max(0, lo - begin), min(tiles[b], hi - begin)
                if t1 > t0:
                    mine.append((b, u, t0, t1, tiles[b]))
        p.segments.append(mine)
    return p


def check(p, lengths, nodes, heads):
    """Every tile of every unit in one part, in order; a part that holds a piece
    of a unit leaves it in a place of its own, and the join adds up just those."""
    k = FEW if p.kernel == "few" else PAIRS
    pieces, places = {}, set()
    for i, mine in enumerate(p.segments):
        for b, u, t0, t1, T in mine:
            pieces.setdefault((b, u), []).append((i, t0, t1))
            if (t0, t1) != (0, T):
                place = 2 * i + (0 if t0 > 0 else 1)
                assert place not in places
                places.add(place)
    joined = set()
    for b, x in enumerate(lengths):
        T = 0 if x is None else up(nodes, k["tile"]) + up(x, k["tile"])
        for u in range(up(nodes * heads, k["rows"])):
            got = pieces.pop((b, u), [])
            assert [t for _, t, _ in got] + [T] == [0] + [t for _, _, t in got], (b, u, got, T)
            if len(got) > 1:
                at = got[1][0]
                assert [i for i, _, _ in got] == list(range(at - 1, at - 1 + len(got))), (b, u, got)
                assert p.cuts.get(at) == (b, u, len(got)), (at, p.cuts.get(at), got)
                joined.add(at)
    assert not pieces and joined == set(p.cuts)
