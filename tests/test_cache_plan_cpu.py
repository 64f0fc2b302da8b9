"""The work lists of the operators on windows, pages and caches made shorter, without a GPU: launches that are only written
down (cache_host.cpp), followed pair by pair.  Every key that a row sees is met once, every partial result joined once,
inside the workspace."""
import contextlib
import ctypes
import os
import random
import subprocess

import pytest

from quantized_decoder_decode_gb300 import build as fqbuild
from quantized_decoder_decode_gb300 import fq

HERE = os.path.dirname(os.path.abspath(__file__))
NAMES = ("fq_attn_window", "fq_attn_window_workspace", "fq_attn_paged", "fq_qk_norm_rope_paged", "fq_attn_key_weights",
         "fq_attn_key_weights_workspace", "fq_kv_evict", "fq_last_error")
P, BIG, TILE, BLOCK = 0x10000, 1 << 40, 128, 96
HEADS = [(4, 4), (4, 2), (8, 2), (8, 1), (16, 8), (32, 4), (3, 3)]


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    fqbuild.build()
    out = os.path.join(str(tmp_path_factory.mktemp("cache_host")), "cache_host.so")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-w", "-fvisibility=default", "-Wl,-Bsymbolic",
                           "-I", fqbuild.INCLUDE, "-I", fqbuild.CSRC, "-I",
                           os.path.join(os.path.dirname(os.path.dirname(fqbuild.NVCC)), "include"), "-x", "c++",
                           os.path.join(HERE, "cache_host.cpp"), "-o", out])
    L, real = ctypes.CDLL(out), fq.lib()
    for n in NAMES:
        getattr(L, n).argtypes, getattr(L, n).restype = getattr(real, n).argtypes, getattr(real, n).restype
    return L


@contextlib.contextmanager
def recorded(L):
    real, fq._lib = fq._lib, L

    def launches():
        out = []
        for i in range(L.cache_host_launches(0)):
            n = L.cache_host_launch(i, None, 0)
            a = (ctypes.c_longlong * n)()
            L.cache_host_launch(i, a, n)
            out.append(list(a))
        L.cache_host_launches(1)
        return out
    try:
        launches()
        yield launches
    finally:
        fq._lib = real


def view(rows, hkv, base=P):
    return fq.fq_kv_view(base, base + (1 << 36), rows, 128, rows * 128)


def visible(i, L, K, window, sinks):
    """The keys that row i sees, as ranges."""
    e = min(K, i + 1 + K - L)
    if e <= 0:
        return []
    lo = max(0, e - window) if window else 0
    s = min(sinks, lo)
    return [r for r in ((0, s), (lo, e)) if r[1] > r[0]]


def tiles_of(window, sinks, K, off, tok, n_tok):
    """Key tiles that rows tok .. tok + n_tok - 1 look at, in order."""
    last = min(K, tok + n_tok - 1 + off)
    if n_tok <= 0 or last <= 0:
        return []
    first = max(0, tok + off - window) // TILE if window else 0
    s = min(-(-min(sinks, last) // TILE), first)
    return list(range(s)) + list(range(first, -(-last // TILE)))


class Window:
    """One call's launches: for every row the key ranges that its finished output is made of."""

    def __init__(self, raw, q_len, k_len, hq, hkv, window, sinks, ws_bytes):
        self.q_len, self.k_len, self.hq, self.hkv, self.G = q_len, k_len, hq, hkv, hq // hkv
        self.window, self.sinks = window, sinks
        self.finished, self.parts, self.most = {}, {}, {False: 0, True: 0}
        for v in raw:
            (self.tiles, self.rows, self.join)[v[0]](v[1:])
        assert not self.parts, f"{len(self.parts)} partial results are never joined"
        assert (self.most[False] * TILE + self.most[True] * 8) * hkv * (128 + 2) * 4 <= ws_bytes

    def done(self, row, keys):
        assert row not in self.finished, f"row {row} is written twice"
        self.finished[row] = keys

    def part(self, small, block, at, row, keys):
        key = (small, block, at)
        assert 0 <= at and at + self.G <= (8 if small else TILE) and key not in self.parts
        self.parts[key] = row, keys
        self.most[small] = max(self.most[small], block + 1)

    def check_mask(self, window, sinks):
        assert (window, sinks) == (self.window or 1 << 30, self.sinks)

    def tiles(self, v):
        room, _, _, hq, hkv, window, sinks, n = v[:8]
        self.check_mask(window, sinks)
        assert 0 < n <= room and (hq, hkv) == (self.hq, self.hkv)
        tpt, seqs = TILE // self.G, v[8 + 4 * n:]
        for i in range(n):
            tok0, info, j0, j1 = v[8 + 4 * i:12 + 4 * i]
            s, single, small, slot = info & 127, info >> 7 & 1, bool(info >> 8 & 1), (info >> 9) - 1
            q_row0, L, _, K, off, _ = seqs[6 * s:6 * s + 6]
            assert L == self.q_len[s] and K == self.k_len[s] and off == K - L + 1
            n_unit = min(L - tok0, tpt if single else 2 * tpt)
            own = tiles_of(self.window, self.sinks, K, off, tok0, n_unit)
            assert 0 <= j0 <= j1 <= len(own)
            for x in range(1 if single else 2):
                for t in range(tok0 + x * tpt, min(L, tok0 + (x + 1) * tpt)):
                    keys = [(j * TILE, (j + 1) * TILE) for j in own[j0:j1]]
                    at = (t - tok0 - x * tpt) * self.G
                    if slot < 0:
                        self.done(q_row0 + t, keys)
                    else:
                        self.part(small, slot + x, at, q_row0 + t, keys)

    def rows(self, v):
        _, hq, hkv, window, sinks, n = v[:6]
        self.check_mask(window, sinks)
        for i in range(n):
            q_row0, n_tok, _, K, off, first, count, block, s = v[6 + 9 * i:15 + 9 * i]
            assert n_tok == self.q_len[s] and K == self.k_len[s]
            last = max(0, min(K, n_tok - 1 + off))
            lo = max(0, off - self.window) // 16 * 16 if self.window else 0
            sn = min(-(-min(self.sinks, last) // 16) * 16, lo) if last else 0
            numbers = (list(range(sn)) + list(range(lo, last)))[first:first + count]
            keys = ranges(numbers)
            for t in range(n_tok):
                if block < 0:
                    self.done(q_row0 + t, keys)
                else:
                    self.part(True, block, t * self.G, q_row0 + t, keys)

    def join(self, v):
        for i in range(v[0]):
            q_row0, n_tok, K, off, a0, nA, a_step, a_row, b0, nB, b_row, c0, nC = v[1 + 13 * i:14 + 13 * i]
            for t in range(n_tok):
                keys = []
                for n, small, first, step, at in ((nA, False, a0, a_step, a_row), (nB, True, b0, 1, b_row), (nC, True, c0, 1, 0)):
                    for p in range(n):
                        row, r = self.parts.pop((small, first + p * step, at + t * self.G))
                        assert row == q_row0 + t
                        keys += r
                self.done(q_row0 + t, keys)


def ranges(numbers):
    out = []
    for k in numbers:
        if out and out[-1][1] == k:
            out[-1][1] = k + 1
        else:
            out.append([k, k + 1])
    return [tuple(r) for r in out]


def covers(got, want, what):
    """The ranges `got` lie apart and hold all of `want`."""
    got = sorted(got)
    for a, b in zip(got, got[1:]):
        assert a[1] <= b[0], f"{what}: keys {b} are met twice"
    for lo, hi in want:
        at = lo
        for a, b in got:
            if a <= at < b:
                at = b
        assert at >= hi, f"{what}: key {at} of {(lo, hi)} is not met"


def check_window(host, q_len, k_len, hq, hkv, window, sinks, paged, own_views=False):
    with recorded(host) as launches:
        ws = fq.fq_attn_window_workspace(q_len, k_len, hq, hkv, window, sinks)
        if paged:
            pages = fq.fq_kv_pages(P, P, 1 << 20, 16, 16 * 128 * hkv, 128, 16 * 128)
            fq.fq_attn_paged(P, pages, P, 1 << 27, q_len, k_len, hq, hkv, window, sinks, 0.1, BIG, P if ws else 0, ws)
        else:
            rows = max(1, sum(k_len))
            views = [view(rows, hkv, P + (s << 42)) for s in range(len(q_len))] if own_views else view(rows, hkv)
            fq.fq_attn_window(P, views, q_len, k_len, hq, hkv, window, sinks, 0.1, BIG, P if ws else 0, ws)
        w = Window(launches(), q_len, k_len, hq, hkv, window, sinks, ws)
    row = 0
    for L, K in zip(q_len, k_len):
        for i in range(L):
            covers(w.finished[row], visible(i, L, K, window, sinks), f"row {i} of {L} over {K}, window {window} {sinks}")
            row += 1
    assert len(w.finished) == row


def length(rng):
    return rng.choice((0, 1, 2, 3, rng.randint(0, 40), rng.randint(0, 300), rng.randint(0, 1500)))


@pytest.mark.parametrize("seed", range(6))
def test_every_visible_key_once(host, seed):
    rng = random.Random(seed)
    for _ in range(60):
        n = rng.choice((1, 1, 2, 3, 5, 18, 64))
        q = [length(rng) for _ in range(n)]
        k = [rng.choice((m, m, m + length(rng), length(rng), m + rng.randint(0, 30000))) for m in q]
        window, sinks = rng.choice((0, 1, 16, 127, 128, 129, rng.randint(1, 3000))), rng.choice((0, 1, 4, 128, rng.randint(0, 400)))
        check_window(host, q, k, *rng.choice(HEADS), window, sinks, rng.random() < .5, rng.random() < .5)


def test_long_beside_many_short(host):
    """Calls with so many units or groups that whole ones fill the SMs: the long one is cut all the same.  And more heads than
    thread blocks."""
    check_window(host, [1, 2, 0, 30], [3000, 64, 5, 100], 1000, 1000, 0, 0, False)
    for q, k in (([1] * 56, [500] * 55 + [30000]), ([20] * 60 + [200], [20] * 60 + [30200]), ([1] * 64, [1] * 63 + [1 << 20])):
        for paged in (False, True):
            check_window(host, q, k, 32, 8, 0, 0, paged)
            check_window(host, q, k, 8, 8, 5000, 7, paged)
    with recorded(host) as launches:   # (one kv head: the most chunks)
        ws = fq.fq_attn_window_workspace([1] * 64, [127] * 63 + [1 << 22], 1, 1, 0, 0)
        fq.fq_attn_window(P, view(1 << 23, 1), [1] * 64, [127] * 63 + [1 << 22], 1, 1, 0, 0, 0.1, BIG, P, ws)
        launches()


def test_largest_lengths(host):
    with recorded(host) as launches:
        for q, k in (([1], [1 << 30]), ([64], [1 << 30]), ([1] * 64, [1 << 30] * 64), ([1 << 24], [1 << 24])):
            for window, sinks in ((0, 0), (1 << 29, 1 << 29), (1000, 4), (2 ** 32 - 1, 2 ** 32 - 1)):
                views = [view(1 << 30, 1, P + (s << 42)) for s in range(len(q))]
                ws = fq.fq_attn_window_workspace(q, k, 8, 1, window, sinks)
                fq.fq_attn_window(P, views, q, k, 8, 1, window, sinks, 0.1, BIG, P, ws)
                for v in launches():
                    assert all(-1 << 31 <= x < 1 << 31 for x in v)


def check_weights(host, q_len, k_len, hq, hkv, window, sinks, own_views):
    with recorded(host) as launches:
        ws = fq.fq_attn_key_weights_workspace(q_len, k_len, hq, hkv, window, sinks)
        rows = max(1, sum(k_len))
        if own_views:
            views = [view(rows, hkv, P + (s << 42)) for s in range(len(q_len))]
            after = [fq.fq_key_weights(BIG + (s << 32), rows) for s in range(len(q_len))]
        else:
            views, after = view(rows, hkv), fq.fq_key_weights(BIG, rows)
        fq.fq_attn_key_weights(P, P, views, q_len, k_len, hq, hkv, window, sinks, 0.1, None, after, P if ws else 0, ws)
        raw = launches()
    G = hq // hkv
    written, met = {}, set()       # (sequence, head, key tile): how often; (sequence, head, key tile, query block)

    def write(s, h, j, more):      # the first time what was there before is added to, then what has been written
        assert more == ((s, h, j) in written), "a key's earlier sums are lost"
        written[s, h, j] = True

    def joined(units, join):
        """One launch: its unfinished sums against the list of those that are joined."""
        parts = {}
        for s, h, kind, more, j0, j1, b0, b1, slot in units:
            if slot >= 0:
                assert kind == 0 and slot not in parts and (slot + 1) * 256 * 4 <= ws
                parts[slot] = s, h, more, j0, j1
        for s, h, more, j0, j1, first, others, n in join:
            for slot in [first] + [others + 2 * i for i in range(n)]:
                assert parts.pop(slot) == (s, h, more, j0, j1)
            for j in range(j0, j1):
                write(s, h, j, more)
        assert not parts, "sums that nobody adds up"

    i = 0
    while i < len(raw):
        v = raw[i]
        assert v[0] == 4 and v[8] <= v[1] and v[7] <= 152 and tuple(v[5:7]) == (window or 1 << 30, sinks)
        units = [tuple(v[10 + 9 * u:19 + 9 * u]) for u in range(v[9])]
        join = []
        if i + 1 < len(raw) and raw[i + 1][0] == 5:
            i += 1
            join = [tuple(raw[i][2 + 8 * e:10 + 8 * e]) for e in range(raw[i][1])]
        i += 1
        for s, h, kind, more, j0, j1, b0, b1, slot in units:
            assert 0 <= j0 < j1 and 0 <= b0 < b1 and b1 - b0 <= 4096
            if kind == 0:
                assert j1 - j0 <= 2
            if kind == 1:
                assert (b0, b1) == (0, 1) and j1 - j0 <= 4096
            for j in range(j0, j1):
                if slot < 0:
                    write(s, h, j, more)
                for b in range(b0, b1) if kind < 2 else ():
                    assert (s, h, j, b) not in met
                    met.add((s, h, j, b))
        joined(units, join)
    for s, (L, K) in enumerate(zip(q_len, k_len)):
        for h in range(hkv):
            for j in range(-(-K // TILE)):
                assert (s, h, j) in written, f"keys of tile {j} of sequence {s} are not written"
        step = max(1, L // 40)
        for i in list(range(0, L, step)) + [L - 1] * (L > 0):
            for lo, hi in visible(i, L, K, window, sinks):
                for j in range(lo // TILE, -(-hi // TILE)):
                    for b in {i * G // BLOCK, (i * G + G - 1) // BLOCK}:
                        for h in {0, hkv // 2, hkv - 1}:
                            assert (s, h, j, b) in met, f"row {i} and key tile {j} of sequence {s} do not meet"


@pytest.mark.parametrize("seed", range(4))
def test_every_key_gets_its_weights_once(host, seed):
    rng = random.Random(50 + seed)
    for _ in range(60):
        n = rng.choice((1, 1, 2, 3, 18, 64))
        q = [length(rng) for _ in range(n)]
        k = [rng.choice((m, m, m + length(rng), length(rng), m + rng.randint(0, 9000))) for m in q]
        window, sinks = rng.choice((0, 1, 16, 128, rng.randint(1, 3000))), rng.choice((0, 1, 4, 128, rng.randint(0, 400)))
        check_weights(host, q, k, *rng.choice(HEADS), window, sinks, rng.random() < .5)


def test_weights_of_long_sequences(host):
    check_weights(host, [8192], [8192], 32, 8, 0, 0, False)
    check_weights(host, [8192], [8192], 32, 8, 1000, 4, False)
    check_weights(host, [1] * 64, [300] * 63 + [60000], 8, 1, 100, 4, True)
    check_weights(host, [70] * 3, [50000] * 3, 32, 4, 0, 0, False)
    check_weights(host, [60000, 1, 50], [500, 600000, 1000], 8, 1, 0, 0, False)    # more query blocks, key tiles than an entry has
    check_weights(host, [400000] * 2, [300, 256], 4, 4, 0, 0, True)
    check_weights(host, [0, 0], [1 << 25, 100], 4, 4, 0, 0, False)
    check_weights(host, [300, 1], [200, 900], 1000, 1000, 0, 0, False)


def test_evict_blocks_and_numbers(host):
    with recorded(host) as launches:
        k_len, keep, hkv = [100, 0, 7, 5000, 1], [50, 9, 7, 700, 0], 3
        n = [min(a, b) for a, b in zip(k_len, keep)]
        fq.fq_kv_evict(view(sum(k_len), hkv), fq.fq_key_weights(P, sum(k_len)), None, k_len, keep, 0, 0, hkv,
                       view(sum(n), hkv, P + (1 << 40)), None, None, P)
        v, = launches()
    assert v[:4] == [6, 5000, 3 * sum(-(-m // 32) for m in n), 5]
    at = blocks = 0
    for i, m in enumerate(n):
        assert v[4 + 4 * i:8 + 4 * i] == [k_len[i], m, at, blocks]
        at, blocks = at + hkv * m, blocks + hkv * -(-m // 32)
