"""What the work lists of the attention operators make of a call: the launches written down by attn_host.cpp,
followed row by row."""
from quantized_decoder_decode_gb300 import fq

P = 0x10000      # made-up addresses, 16-byte aligned
BIG = 1 << 40
TILE = 128


def view(base, rows, hkv):
    return fq.fq_kv_view(base, base + (1 << 36), rows, 128, rows * 128)


class Launches:
    """The launches of one call: finished[row] is a list of (source, first key, last key + 1), where the source is
    the sequence whose keys they are (n_seq: the shared prefix); asserts on the way that no partial result is
    written twice, read for another row, or lost, and that no list passes its bounds."""

    def __init__(self, raw, hq, hkv, ws_bytes, views, source_of):
        self.hq, self.hkv, self.G = hq, hkv, hq // hkv
        self.views, self.source_of = views, source_of
        self.finished, self.parts, self.reached = {}, {}, []
        self.most = {False: 0, True: 0}   # partial blocks of 128 and of 8 rows
        for v in raw:
            (self.tiles, self.rows, self.join)[v[0]](v[1:])
        assert not self.parts, f"{len(self.parts)} partial results are never joined"
        # values and (m, l) of each block
        need = (self.most[False] * TILE + self.most[True] * 8) * hkv * (128 + 2) * 4
        assert need <= ws_bytes, (need, ws_bytes)

    def done(self, row, ranges):
        assert row not in self.finished, f"row {row} is written twice"
        self.finished[row] = [r for r in ranges if r[2] > r[1]]

    def part(self, small, block, at, row, r):
        assert 0 <= at and at + self.G <= (8 if small else TILE)
        key = (small, block, at)
        assert key not in self.parts, f"partial result {key} is written twice"
        self.parts[key] = row, r
        self.most[small] = max(self.most[small], block + 1)

    def tiles(self, v):
        room, n_views, hq, hkv, n = v[:5]
        assert (hq, hkv) == (self.hq, self.hkv) and 0 < n <= room
        self.reached.append(("tiles", room, n_views, n))
        e, s = v[5:5 + 4 * n], v[5 + 4 * n:5 + 4 * n + 6 * 65]
        maps = v[5 + 4 * n + 6 * 65:]
        assert len(maps) == 8 * n_views
        tpt = TILE // self.G
        for i in range(n):
            tok0, info, j0, j1 = e[4 * i:4 * i + 4]
            seq, single, small, slot = info & 127, info >> 7 & 1, bool(info >> 8 & 1), (info >> 9) - 1
            q_row0, q_len, k_row0, k_len, off, w = s[6 * seq:6 * seq + 6]
            assert q_len > tok0 and j0 <= j1 and 0 <= w < n_views
            if j1 > j0:
                src = self.source_of(seq)
                want = self.views[src]
                kb, krows, krs, khs, vb, vrows, vrs, vhs = maps[8 * w:8 * w + 8]
                assert (kb, vb) == (want.k, want.v) and krows == vrows and k_row0 + k_len <= krows <= want.rows
                assert (krs, vrs) == (2 * want.row_stride,) * 2
                assert hkv == 1 or (khs, vhs) == (2 * want.head_stride,) * 2
            for x in range(1 if single else 2):
                for t in range(tok0 + x * tpt, min(q_len, tok0 + (x + 1) * tpt)):
                    r = (self.source_of(seq), j0 * TILE, min(j1 * TILE, max(0, min(k_len, t + off))))
                    if slot < 0:
                        self.done(q_row0 + t, [r])
                    else:
                        self.part(small, slot + x, (t - tok0 - x * tpt) * self.G, q_row0 + t, r)

    def rows(self, v):
        beside, hq, hkv, n = v[:4]
        assert (hq, hkv) == (self.hq, self.hkv) and 0 < n <= 3 * 152 + 65
        self.reached.append(("rows", beside, n))
        for i in range(n):
            q_row0, n_tok, k_row0, k_len, off, first, chunk, slot, k, vv = v[4 + 10 * i:14 + 10 * i]
            assert n_tok * self.G <= 8 and chunk > 0 and chunk % 64 == 0
            src = [s for s, w in self.views.items() if (w.k, w.v) == (k, vv)] if k_len else [0]
            for t in range(n_tok):
                limit = max(0, min(k_len, t + off))
                r = (self.row_source(src, q_row0, k_row0, k_len), first, max(first, min(first + chunk, limit)))
                if slot < 0:
                    self.done(q_row0 + t, [r])
                else:
                    self.part(True, slot, t * self.G, q_row0 + t, r)

    def row_source(self, candidates, q_row0, k_row0, k_len):
        return candidates[0] if len(candidates) == 1 else self.source_of((candidates, q_row0, k_row0, k_len))

    def join(self, v):
        room, n, max_tok, max_parts = v[:4]
        assert 0 < n <= room
        self.reached.append(("join", room, n))
        for i in range(n):
            q_row0, n_tok, k_len, off, a0, nA, a_step, a_row, b0, nB, b_row, c0, nC = v[4 + 13 * i:17 + 13 * i]
            assert 0 < n_tok <= max_tok and nA + nB + nC <= max_parts
            for t in range(n_tok):
                at = [(False, a0 + p * a_step, a_row + t * self.G) for p in range(nA)] + \
                     [(True, b0 + p, b_row + t * self.G) for p in range(nB)] + [(True, c0 + p, t * self.G) for p in range(nC)]
                got = [self.parts.pop(k) for k in at]
                assert all(row == q_row0 + t for row, _ in got)
                ranges = [r for _, r in got]
                assert (min(k_len, t + off) > 0) == any(r[2] > r[1] for r in ranges)
                self.done(q_row0 + t, ranges)


def covers(ranges, want):
    """The ranges of one row, put together, are [0, n) of every source in want, each key once."""
    left = dict(want)
    at = dict.fromkeys(want, 0)
    for src, lo, hi in sorted(ranges):
        if at.get(src) != lo:
            return False
        at[src] = hi
    return all(at[s] == n for s, n in left.items())


def prompt(launches, q_len, k_len, hq, hkv, own_views):
    """One fq_attn_prompt call followed through; the kinds of launches that it made."""
    n = len(q_len)
    need = fq.fq_attn_prompt_workspace(q_len, k_len, hq, hkv)
    k0 = [0] * n if own_views else [sum(k_len[:s]) for s in range(n)]
    if own_views:
        views = {s: view(P + s * BIG, max(1, k_len[s]), hkv) for s in range(n)}
        arg = [views[s] for s in range(n)]
    else:
        arg = view(P, max(1, sum(k_len)), hkv)
        views = {s: arg for s in range(n)}
    q0 = [sum(q_len[:s]) for s in range(n)]

    def source(x):   # a sequence, or (sequences of one view, first query row, first key row, keys)
        if not isinstance(x, tuple):
            return x
        return next(s for s in x[0] if q_len[s] and (q0[s], k0[s], k_len[s]) == x[1:])
    launches()
    fq.fq_attn_prompt(P, arg, q_len, k_len, hq, hkv, 0.1, P, P, need)
    got = Launches(launches(), hq, hkv, need, views, source)
    for s in range(n):
        for t in range(q_len[s]):
            seen = max(0, min(k_len[s], t + k_len[s] - q_len[s] + 1))
            assert covers(got.finished.pop(q0[s] + t), {s: seen} if seen else {}), (s, t)
    assert not got.finished
    return got.reached


def shared(launches, prefix_len, tail_len, hq, hkv):
    n = len(tail_len)
    need = fq.fq_attn_shared_workspace(prefix_len, tail_len, hq, hkv)
    views = {s: view(P + s * BIG, max(1, t), hkv) for s, t in enumerate(tail_len)}
    views[n] = view(P + n * BIG, max(1, prefix_len), hkv)
    launches()
    fq.fq_attn_shared(P, views[n], prefix_len, [views[s] for s in range(n)], tail_len, hq, hkv, 0.1, P, P, need)
    got = Launches(launches(), hq, hkv, need, views, lambda s: s)
    for s in range(n):
        want = {k: v for k, v in ((s, tail_len[s]), (n, prefix_len)) if v}
        assert covers(got.finished.pop(s), want), s
    assert not got.finished
    return got.reached


# Calls that need the larger parameter blocks, or lists longer than one launch takes: (query lengths, key lengths, query
# heads, kv heads, a view per sequence, the launches that it takes as (kind, entries or items)).  Heads of 8 / 1
# make a tile 16 tokens.
MANY = {
    "many views": ([20 + i % 21 for i in range(40)], [20 + i % 21 + (37 * i % 90) for i in range(40)], 8, 2, True,
                   [("tiles", 768)]),
    "many entries over several views": ([333, 2000, 900], [333, 2100, 3000], 8, 1, True, [("tiles", 768)]),
    "two launches over several views": ([400] * 64, [400 + 7 * (i % 5) for i in range(64)], 8, 1, True,
                                        [("tiles", 768), ("tiles", 768)]),
    "two launches over one view": ([800] * 64, [800] * 64, 8, 1, False, [("tiles", 1536), ("tiles", 1536)]),
    "two launches beside single tokens": ([450] * 60 + [1] * 4, [450] * 60 + [9000, 3000, 1500, 5], 8, 1, True,
                                          [("tiles", 768), ("tiles", 768), ("rows",), ("join", 64)]),
    "many joins": ([2000], [20000], 8, 1, False, [("tiles", 1536), ("join", 512)]),
    "many joins of many parts": ([600] + [1] * 40, [60000] + [5000] * 40, 8, 1, True, [("tiles", 1536), ("rows",), ("join", 512)]),
    "two launches of joins": ([9920], [20000], 8, 1, False, [("tiles", 1536), ("join", 512), ("join", 512)]),
}
