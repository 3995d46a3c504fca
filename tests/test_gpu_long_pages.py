"""GPU tests of 4-bit pages, windows with first tokens, and positions of several
axes, against the plain 64-bit forms in longhelp.py.  Weights enter the value
product as two bf16 (2^-17 of each term that they multiply).  A 4-bit value q s + z is the
terms (q - c) s and z + c s: beside 8-bit keys c is the integer nearest to -z / s, so that
their magnitudes add up to at most 3 |v|; beside 4-bit keys it is 8, and they add up to at
most |v - (z + 8 s)| + |z + 8 s| <= 8 s + |z + 8 s| (q <= 15: |q - 8| <= 8).  So the error is
2^-17 of sum p times 3 |v|, or times that sum."""
import math

import numpy as np
import pytest
import torch

import agent_shared_compressed_gb300 as kv
from agent_shared_compressed_gb300 import build as kvbuild
from agent_shared_compressed_gb300 import synth
import longhelp as Lg
import pageshelp as P
from kvhelp import Guarded

pytestmark = pytest.mark.gpu
FMTS = ["bf16", "k8v8", "k8v4", "k4v4"]
WEIGHTS = 3 * 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def built():
    kvbuild.build()
    kv.load()


def _kv(n, H, d, seed):
    k, v = synth.kv_layer(H, max(n, 1), d, torch.Generator().manual_seed(seed))
    return k.transpose(0, 1)[:n].contiguous().cuda(), v.transpose(0, 1)[:n].contiguous().cuda()


def _case(fmt, H, d, page, lens, G, m, window, sinks, seed=0, base=False, forget=True, max_pages=None, scale=None, plain=False):
    """Writes random sequences, attends and compares."""
    rng = np.random.default_rng(seed + 1)
    pg = Lg.Pages(fmt, H, d, page, lens, seed=seed, max_pages=max_pages)
    k, v = _kv(sum(lens), H, d, seed)
    if sum(lens):
        pg.write(k, v)
    if forget and window:
        pg.forget(m, window, sinks)
    hk, hv = Lg.held(Lg.f64(k), fmt, False), Lg.held(Lg.f64(v), fmt, True)
    q = Lg.bf16(rng.standard_normal((len(lens), m, H * G, d))).cuda()
    scale = 1 / math.sqrt(d) if scale is None else scale
    bo = bl = None
    if base:
        bo = torch.from_numpy(0.1 * rng.standard_normal(q.shape)).float().cuda()
        bl = torch.from_numpy(rng.uniform(2, 6, q.shape[:3])).float().cuda()
        bl[0, 0, 0] = -math.inf
    out, lse = pg.attend(q, scale, window, sinks, bo, bl, plain=plain)
    assert pg.status() == kv.KVP_OK
    for b, (kb, vb) in enumerate(zip(Lg.split(hk, lens), Lg.split(hv, lens))):
        ro, rl, mass, reach = Lg.rows(Lg.f64(q[b]), kb, vb, [lens[b] - m + i for i in range(m)], window, sinks, scale,
                                      2 * Lg.zero_points(kb) if fmt == "k4v4" and lens[b] else None)
        if base:
            ro, rl, mass = Lg.join(ro, rl, mass, bo[b].cpu().numpy().astype(np.float64), bl[b].cpu().numpy().astype(np.float64))
        if fmt == "k4v4" and lens[b]:
            mass = _middle_mass(Lg.f64(q[b]), kb, vb, [lens[b] - m + i for i in range(m)], window, sinks, scale, mass)
        Lg.check(out[b], lse[b], ro, rl, mass, reach, WEIGHTS)


def _middle_mass(q, k, v, places, window, sinks, scale, mass):
    """sum p (8 s + |z + 8 s|) / 3 of 4-bit values (as large as WEIGHTS wants it), at least sum p |v|.
    s, z from the held values: their group's least and (at most) largest."""
    g = v.reshape(*v.shape[:-1], -1, 32)
    s, z = (g.max(-1, keepdims=True) - g.min(-1, keepdims=True)) / 15, g.min(-1, keepdims=True)
    terms = np.repeat(8 * s + np.abs(z + 8 * s), 32, -1).reshape(v.shape) * (1 + 2.0 ** -9)
    return np.maximum(mass, Lg.rows(q, k, terms, places, window, sinks, scale)[0] / 3)


# --- 4-bit pages ---------------------------------------------------------------

@pytest.mark.parametrize("H,d,page,lens", [(1, 128, 16, [1]), (3, 64, 16, [0, 37, 16, 1]), (8, 128, 64, [130, 15]),
                                           (2, 128, 1024, [1025]), (5, 64, 128, [200, 0])])
def test_4bit_write_and_read_back_exact(H, d, page, lens):
    """Unrotated rows: what the pages hold is the format's definition, bit for bit."""
    pg = Lg.Pages("k4v4", H, d, page, lens, L=2, layer=1, seed=d + H)
    k, v = _kv(sum(lens), H, d, 7)
    k[0, 0, :32] = 1.5                                     # a constant group: scale 0
    if d == 128:
        k[0, 0, 32:64] = 0.0
    ko, vo = pg.write(k, v)
    hk, hv = P.to_bf16(P.held4(Lg.f64(k))), P.to_bf16(P.held4(Lg.f64(v)))
    assert np.array_equal(ko, hk) and np.array_equal(vo, hv)
    rk, rv = pg.read(max(lens) + 3)
    for b, (x, y) in enumerate(zip(Lg.split(hk, lens), Lg.split(hv, lens))):
        assert np.array_equal(rk[b].transpose(1, 0, 2)[:lens[b]], x) and np.array_equal(rv[b].transpose(1, 0, 2)[:lens[b]], y)
        assert not rk[b][:, lens[b]:].any() and not rv[b][:, lens[b]:].any()
    assert pg.status() == kv.KVP_OK


@pytest.mark.parametrize("fmt", ["k8v8", "k8v4", "k4v4"])
@pytest.mark.parametrize("d", [64, 128])
def test_codes_at_every_border(fmt, d):
    """Halves of codes and their neighbours (in 16 bits ties are common), scales that are 0,
    the smallest, subnormal and held at the largest, zero points far from the range: bit for bit."""
    rng = np.random.default_rng(d)
    rows = [np.full(d, 2.0 ** -26), 2.0 ** -26 * rng.choice([-1.0, 1.0], d), 2.0 ** -19 * rng.standard_normal(d),
            3e38 * rng.uniform(-1, 1, d), np.where(np.arange(d) % 32 == 7, 3e38, rng.standard_normal(d))]
    for size in (0.0, 1.0, -100.0, 6e4):                  # the middle, beside a range of about 4
        rows += [size + x for x in rng.standard_normal((300, d))]
    for scale in 2.0 ** np.arange(-24, 11, 3.0):          # whole codes, halves and what lies next to them
        for top, off in ((127.0, -64.0), (15.0, 0.0)):
            x = scale * (rng.integers(0, int(top), (20, d)) + rng.choice([0.0, 0.5, 0.5 - 2.0 ** -7, 0.5 + 2.0 ** -7], (20, d)) + off)
            x[:, ::32], x[:, 1::32] = scale * top, scale * off
            rows += list(x)
    x = Lg.bf16(np.stack(rows)[:, None]).cuda()
    pg = Lg.Pages(fmt, 1, d, 32, [x.shape[0]])
    ko, vo = pg.write(x, x.neg())
    held = {"k8v8": (Lg.held8, Lg.held8), "k8v4": (Lg.held8, P.held4), "k4v4": (P.held4, P.held4)}[fmt]
    assert np.array_equal(ko, P.to_bf16(held[0](Lg.f64(x))))
    assert np.array_equal(vo, P.to_bf16(held[1](-Lg.f64(x))))


def test_4bit_keys_are_coded_from_the_turned_fp32_key():
    """Half a step of the group's range, (max - min) / 30 (its scale rounded to fp16:
    15 codes' worth of 2^-11 of it; the zero point 2^-11 of itself), fp32 angles and
    turn (2^-19 of the pair's norm), and a bf16 rounding on the way out."""
    H, d, n = 2, 128, 75
    pg = Lg.Pages("k4v4", H, d, 16, [n])
    k, v = _kv(n, H, d, 3)
    pos = torch.arange(1 << 20, (1 << 20) + n, device="cuda")
    freq = [500000.0 ** (-2.0 * i / d) for i in range(d // 2)]
    ko, vo = (Guarded(n * H * d * 2) for _ in range(2))
    assert kv.kvpages_append(pg.buf.t, pg.cfg, 0, n, 0, None, k, v, pg.slots, pos, None, None, 0.0, d, freq, None, ko.t,
                             vo.t) == kv.KVP_OK
    want = P.heads(Lg.f64(k), None, 0.0, pos.cpu().numpy(), freq, d)
    g = want.reshape(n, H, -1, 32)
    lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
    pair = np.abs(want).max(-1, keepdims=True)[..., None] * 2.0 ** -17
    tol = (hi - lo) / 30 + (hi - lo) * 2.0 ** -11 + np.abs(lo) * 2.0 ** -11 + pair + 2.0 ** -8 * (np.abs(g) + (hi - lo) / 15)
    assert np.all(np.abs(Lg.f64(ko.bf16((n, H, d))).reshape(g.shape) - g) <= tol)
    assert np.array_equal(Lg.f64(vo.bf16((n, H, d))), P.to_bf16(P.held4(Lg.f64(v))))


def test_4bit_nonfinite_and_range():
    """Inf and NaN keys count and code as zeros and are reported; a range beyond fp16 is
    held at its largest scale."""
    pg = Lg.Pages("k4v4", 1, 64, 16, [3])
    k, v = _kv(3, 1, 64, 1)
    bad = k.clone()
    bad[1, 0, 3], bad[1, 0, 40] = math.inf, math.nan
    ko, _ = pg.write(bad, v)
    assert pg.status() == kv.KVP_ERR_NONFINITE
    clean = Lg.f64(bad)
    clean[~np.isfinite(clean)] = 0
    assert np.array_equal(ko, P.to_bf16(P.held4(clean)))
    pg = Lg.Pages("k4v4", 1, 64, 16, [3])
    k[2, 0, 5] = 1e30
    ko, _ = pg.write(k, v)
    assert pg.status() == kv.KVP_ERR_RANGE and np.array_equal(ko, P.to_bf16(P.held4(Lg.f64(k))))


@pytest.mark.parametrize("H,G,d,page,lens,m", [
    (1, 1, 128, 16, [1], 1), (1, 4, 64, 16, [0, 3, 31, 33], 1), (8, 4, 128, 64, [700, 0, 129], 1),
    (2, 8, 128, 16, [333, 18], 1), (4, 3, 64, 128, [513, 40, 7, 256], 5), (2, 4, 128, 32, [90, 2], 16), (1, 1, 64, 16, [5000], 64),
    (3, 5, 128, 64, [4096, 1], 2), (32, 1, 64, 32, [180, 0, 99, 1, 15, 17], 1)])
@pytest.mark.parametrize("roomy", [False, True])
def test_4bit_attention(H, G, d, page, lens, m, roomy):
    """Head layouts, row counts of every tile, lengths from none, teams and runs."""
    _case("k4v4", H, d, page, lens, G, m, 0, 0, seed=H * 7 + m, max_pages=20000 // page if roomy else None, plain=True)


def test_4bit_attention_joined_and_sharp():
    """With a base; and with scores spread over hundreds."""
    _case("k4v4", 4, 128, 16, [600, 31, 0], 4, 2, 0, 0, base=True, plain=True)
    _case("k4v4", 4, 64, 16, [600, 31, 0], 2, 1, 0, 0, scale=2.0, plain=True)


def test_4bit_zero_points_far_from_zero():
    """Keys whose groups lie far from zero (a constant added to every key): scores differ
    by the codes' part alone, beside a zero part 2^9 as large."""
    rng = np.random.default_rng(5)
    H, d, n = 1, 128, 300
    pg = Lg.Pages("k4v4", H, d, 16, [n])
    k = Lg.bf16(64.0 + 0.5 * rng.integers(0, 16, (n, H, d))).cuda()
    _, v = _kv(n, H, d, 2)
    pg.write(k, v)
    hk, hv = P.held4(Lg.f64(k)), P.held4(Lg.f64(v))
    q = Lg.bf16(rng.standard_normal((1, 1, 4, d))).cuda()
    out, lse = pg.attend(q, 0.1)
    ro, rl, mass, reach = Lg.rows(Lg.f64(q[0]), hk, hv, [n - 1], 0, 0, 0.1, 2 * Lg.zero_points(hk))
    mass = _middle_mass(Lg.f64(q[0]), hk, hv, [n - 1], 0, 0, 0.1, mass)
    Lg.check(out[0], lse[0], ro, rl, mass, reach, WEIGHTS)


def test_4bit_large_queries():
    """Queries up to bf16's largest over keys so small that scores are finite; and tiny ones."""
    rng = np.random.default_rng(9)
    H, d, n = 1, 128, 40
    for size, keys, scale in ((3e38, 1e-6, 1e-33), (1e-38, 1.0, 1e37)):
        pg = Lg.Pages("k4v4", H, d, 16, [n])
        k = Lg.bf16(keys * rng.standard_normal((n, H, d))).cuda()
        _, v = _kv(n, H, d, 2)
        pg.write(k, v)
        hk, hv = P.held4(Lg.f64(k)), P.held4(Lg.f64(v))
        q = Lg.bf16(size * rng.uniform(-1, 1, (1, 1, 4, d))).cuda()
        out, lse = pg.attend(q, scale)
        ro, rl, mass, reach = Lg.rows(Lg.f64(q[0]), hk, hv, [n - 1], 0, 0, scale, 2 * Lg.zero_points(hk))
        Lg.check(out[0], lse[0], ro, rl, _middle_mass(Lg.f64(q[0]), hk, hv, [n - 1], 0, 0, scale, mass), reach, WEIGHTS)


# --- windows ---------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H,G,d,page,lens,m,window,sinks", [
    (1, 1, 128, 16, [1, 40], 1, 1, 0), (2, 4, 128, 16, [300, 17, 0, 64], 1, 33, 4), (2, 4, 64, 16, [300, 17, 0, 64], 1, 48, 0),
    (1, 8, 128, 64, [1000, 129], 1, 100, 70), (2, 2, 64, 32, [777, 5, 31], 5, 64, 1), (2, 4, 128, 16, [513, 3], 16, 7, 19),
    (1, 1, 64, 16, [2000], 64, 20, 33), (8, 4, 128, 16, [4096] * 3, 1, 1024, 4), (4, 3, 64, 128, [513, 40, 7, 256], 5, 300, 300)])
def test_window(fmt, H, G, d, page, lens, m, window, sinks):
    """Windows from one token to more than there are, first tokens from none to past the
    window's start; pages that nobody sees are out of the table."""
    _case(fmt, H, d, page, lens, G, m, window, sinks, seed=window + sinks)


@pytest.mark.parametrize("fmt", ["bf16", "k4v4"])
def test_window_joined_runs_and_roomy_tables(fmt):
    _case(fmt, 4, 128, 16, [700, 31, 0], 4, 2, 100, 5, base=True)
    _case(fmt, 2, 128, 64, [9000, 8191], 4, 1, 6000, 4)                        # runs, joined by a second launch
    _case(fmt, 2, 64, 16, [300, 20], 4, 1, 50, 4, max_pages=3000)


@pytest.mark.parametrize("fmt", FMTS)
def test_window_wider_than_everything_is_none(fmt):
    """A window of 2^31 - 1 (and as many first tokens) is no window, bit for bit."""
    lens, H, d = [300, 0, 31], 2, 128
    pg = Lg.Pages(fmt, H, d, 16, lens)
    k, v = _kv(sum(lens), H, d, 4)
    pg.write(k, v)
    q = Lg.bf16(np.random.default_rng(0).standard_normal((3, 3, 8, d))).cuda()
    out, lse = pg.attend(q, 0.1, plain=True)
    big = 2 ** 31 - 1
    for w, s in ((0, 0), (0, 5), (big, 0), (big, big), (300, 0), (1, big)):
        o, l = pg.attend(q, 0.1, w, s)
        assert np.array_equal(o, out) and np.array_equal(l, lse), (w, s)


def test_window_leaves_unseen_values_out():
    """Inf and NaN keys and values between the first tokens and the window, in the blocks
    at its borders too, have no part; one that is seen has one in its dim."""
    H, d, n, window, sinks = 2, 128, 200, 37, 5
    for d in (64, 128):
        pg = Lg.Pages("bf16", H, d, 16, [n])
        k, v = _kv(n, H, d, 6)
        q = Lg.bf16(np.random.default_rng(1).standard_normal((1, 1, 4, d))).cuda()
        pg.write(k, v)
        clean = pg.attend(q, 0.1, window, sinks)
        for x in (k, v):
            x[sinks:n - window] = math.nan
            x[sinks + 1:n - window:3] = math.inf
        pg.write(k, v)
        dirty = pg.attend(q, 0.1, window, sinks)
        assert np.array_equal(clean[0], dirty[0]) and np.array_equal(clean[1], dirty[1])
        v[n - window, 1, 3] = math.inf
        pg.write(k, v)
        out, _ = pg.attend(q, 0.1, window, sinks)
        assert np.all(np.isinf(out[0, 0, 2:, 3])) and np.isinf(out).sum() == 2 and not np.isnan(out).any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,G,page,lens,m,window,sinks,roomy", [
    (2, 4, 16, [200, 3, 90], 1, 37, 5, False), (1, 1, 64, [333, 61], 1, 50, 33, True),         # tiles of 4 rows
    (1, 8, 32, [150, 40], 1, 21, 0, True), (2, 4, 64, [777, 64, 31], 2, 100, 7, False),        # of 8
    (1, 8, 16, [300, 129], 2, 19, 3, False), (2, 3, 128, [513, 40, 256], 5, 77, 40, True),     # of 16
    (1, 1, 16, [2000], 64, 20, 33, False), (1, 4, 64, [9000, 8191], 1, 6001, 9, False)])
def test_window_over_tokens_never_written(fmt, d, H, G, page, lens, m, window, sinks, roomy):
    """Tokens that no query sees are not written at all (a negative slot): the NaN patterns that
    lie in their places, in blocks that hold seen tokens too, have no part.  The result is that of
    pages which hold every token, bit for bit."""
    k, v = _kv(sum(lens), H, d, m + d)
    q = Lg.bf16(np.random.default_rng(G).standard_normal((len(lens), m, H * G, d))).cuda()
    unseen = torch.tensor([sinks <= t < n - (m - 1) - window for n in lens for t in range(n)], device="cuda")
    assert bool(unseen.any())
    got = []
    for leave_out in (False, True):
        pg = Lg.Pages(fmt, H, d, page, lens, max_pages=20000 // page if roomy else None)
        if leave_out:
            pg.slots[unseen] = -1
        pg.write(k, v)
        got.append(pg.attend(q, 1 / math.sqrt(d), window, sinks))
        assert pg.status() == kv.KVP_OK
    assert np.array_equal(got[0][0], got[1][0]) and np.array_equal(got[0][1], got[1][1])


@pytest.mark.parametrize("fmt", ["bf16", "k8v4", "k4v4"])
@pytest.mark.parametrize("past", [1, 2, 5, 16, 32, 33])
def test_lengths_up_to_the_largest(fmt, past):
    """A sequence of 2^31 - past tokens, all of them in one shared page but the last ones, behind
    which nothing has been written: its newest tokens by a window, and all of it."""
    H, d, page, window, sinks = 1, 64, 1024, 70, 3
    pg = Lg.Pages(fmt, H, d, page, [page, page])
    k, v = _kv(2 * page, H, d, past)
    shared, last = (int(pg.table[b, 0]) for b in (0, 1))
    pg.slots[2 * page - past:] = -1
    pg.write(k, v)
    pg.max_pages, pg.lens = 1 << 21, [2 ** 31 - past]
    pg.table_d = torch.full((1, 1 << 21), shared, dtype=torch.int32, device="cuda")
    pg.table_d[0, -1] = last
    pg.lens_d = torch.tensor(pg.lens, dtype=torch.int32, device="cuda")
    hk, hv = Lg.held(Lg.f64(k), fmt, False), Lg.held(Lg.f64(v), fmt, True)
    q = Lg.bf16(np.random.default_rng(past).standard_normal((1, 2, 4, d))).cuda()
    out, lse = pg.attend(q, 0.1, window, sinks)
    n = 2 * page - past                                                        # as two pages: the same tokens are seen
    ro, rl, mass, reach = Lg.rows(Lg.f64(q[0]), hk[:n], hv[:n], [n - 2, n - 1], window, sinks, 0.1,
                                  2 * Lg.zero_points(hk[:n]) if fmt == "k4v4" else None)
    if fmt == "k4v4":
        mass = _middle_mass(Lg.f64(q[0]), hk[:n], hv[:n], [n - 2, n - 1], window, sinks, 0.1, mass)
    Lg.check(out[0], lse[0], ro, rl, mass, reach, WEIGHTS)
    if past == 5:
        # the shared page's tokens, 2^21 - 1 times: a warp adds some 2^16 weights one after the other
        # (2^-24 of half of their sum each, on average, if all are cut to one side: 2^-9)
        out, lse = pg.attend(q, 0.1, 0, 0, plain=True)
        ro, rl, mass, reach = Lg.rows(Lg.f64(q[0]), hk[:page], hv[:page], [page] * 2, 0, 0, 0.1)
        assert np.all(np.abs(out[0] - ro) <= 2.0 ** -6 * np.abs(v.float().cpu().numpy()).max())
        assert np.all(np.abs(lse[0] - rl - 21 * math.log(2)) <= 2.0 ** -8)
    assert pg.status() == kv.KVP_OK


def test_window_in_a_graph_on_another_stream():
    """Captured once, replayed as the sequence grows past its window; another stream than
    the current one, beside a second graph with a workspace of its own."""
    H, d, n, window, sinks = 2, 128, 120, 40, 3
    pg = Lg.Pages("k4v4", H, d, 16, [n])
    k, v = _kv(n, H, d, 8)
    pg.write(k, v)
    hk, hv = P.held4(Lg.f64(k)), P.held4(Lg.f64(v))
    q = Lg.bf16(np.random.default_rng(2).standard_normal((1, 1, 4, d))).cuda()
    st = torch.cuda.Stream()
    calls = []
    for w, s in ((window, sinks), (17, 0)):
        wsb = kv.kvpages_attend_workspace_bytes(pg.cfg, 1, 1, 4)
        ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty(1, 1, 4, d, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 1, 4, device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            kv.check(kv.kvpages_attend_window(pg.buf.t, pg.cfg, 0, 1, 1, 4, q, 0.1, w, s, pg.table_d, pg.max_pages, pg.lens_d,
                                              None, None, out, lse, ws, wsb, torch.cuda.current_stream()))
        calls.append((g, w, s, out, lse, ws))
    for length in (1, 16, 39, 41, 44, 77, 120, 0):
        pg.lens_d.fill_(length)
        torch.cuda.synchronize()
        for g, *_ in calls:
            g.replay()
        torch.cuda.synchronize()
        for _, w, s, out, lse, _ in calls:
            ro, rl, mass, reach = Lg.rows(Lg.f64(q[0]), hk[:length], hv[:length], [length - 1], w, s, 0.1,
                                          2 * Lg.zero_points(hk[:length]) if length else None)
            if length:
                mass = _middle_mass(Lg.f64(q[0]), hk[:length], hv[:length], [length - 1], w, s, 0.1, mass)
            Lg.check(Lg.f64(out[0]), lse[0].cpu().numpy().astype(np.float64), ro, rl, mass, reach, WEIGHTS)


# --- positions with several axes -----------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,rot,n_axes", [(128, 128, 3), (128, 64, 2), (64, 64, 4), (64, 64, 1)])
def test_axes(fmt, d, rot, n_axes):
    """Each axis alone: the pairs of the axis are those of a plain write at its positions,
    bit for bit, queries as well as keys (bf16 pages), for sections and axes in turn; and
    against 64 bits at far positions."""
    H, nq, n = 2, 6, 29
    rng = np.random.default_rng(d + rot)
    x = Lg.bf16(rng.standard_normal((n, nq + 2 * H, d))).cuda()
    pos = torch.from_numpy(rng.integers(-5, 1 << 33, (n_axes, n))).cuda()
    pos[:, 0] = 0
    norm = Lg.bf16(rng.uniform(0.5, 1.5, d)).cuda()
    freq = [500000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]

    def write(call, positions, *more):
        pg = Lg.Pages(fmt, H, d, 16, [n])
        qo, ko, vo = Guarded(n * nq * d * 2), Guarded(n * H * d * 2), Guarded(n * H * d * 2)
        rc = call(pg.buf.t, pg.cfg, 0, n, nq, x[:, :nq], x[:, nq:nq + H], x[:, nq + H:], pg.slots, positions, *more, norm, None,
                  1e-6, rot, freq, qo.t, ko.t, vo.t)
        assert rc == kv.KVP_OK
        torch.cuda.synchronize()
        assert pg.buf.canary_ok() and pg.status() == kv.KVP_OK and all(o.canary_ok() for o in (qo, ko, vo))
        read = pg.read()
        return [Lg.f64(o.bf16((n, h, d))) for o, h in ((qo, nq), (ko, H), (vo, H))] + [read[0], read[1]]

    half = rot // 2
    alone = [write(kv.kvpages_append, pos[a].contiguous()) for a in range(n_axes)]
    for axes in ([i * n_axes // half for i in range(half)], [i % n_axes for i in range(half)], [n_axes - 1] * half):
        got = write(kv.kvpages_append_axes, pos, n_axes, axes)
        of = np.array([axes[i % half] if i < rot else 0 for i in range(d)])
        want = np.choose(of, [alone[a][0] for a in range(n_axes)])
        assert np.array_equal(got[0], want)
        if fmt == "bf16":
            assert np.array_equal(got[1], np.choose(of, [alone[a][1] for a in range(n_axes)]))
        assert np.array_equal(got[2], alone[0][2]) and np.array_equal(got[4], alone[0][4])
        assert np.array_equal(got[3][0].transpose(1, 0, 2), got[1])
        # 64 bits: the angle from exact products (positions below 2^33, frequencies fp32)
        ang = np.stack([np.asarray(pos[axes[i]].cpu().numpy(), np.longdouble) * np.longdouble(np.float32(freq[i]))
                        for i in range(half)], 1)
        c, s = np.cos(ang).astype(np.float64)[:, None], np.sin(ang).astype(np.float64)[:, None]
        y = Lg.f64(x[:, :nq])
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + 1e-6) * Lg.f64(norm)
        a, b = y[..., :half].copy(), y[..., half:rot].copy()
        y[..., :half], y[..., half:rot] = a * c - b * s, b * c + a * s
        size = np.zeros_like(y)
        size[..., :half] = size[..., half:rot] = np.hypot(a, b)
        assert np.all(np.abs(got[0] - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -18 * (size + np.abs(y)))


def test_axes_that_agree_are_one():
    """Text: all axes at the same positions give the plain write's bytes."""
    H, d, n = 3, 128, 40
    k, v = _kv(n, H, d, 1)
    pos = torch.arange(100, 100 + n, device="cuda")
    freq = [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]
    images = []
    for three in (False, True):
        pg = Lg.Pages("k4v4", H, d, 16, [n])
        more = (pos.repeat(3).view(3, n), 3, [i % 3 for i in range(64)]) if three else (pos,)
        call = kv.kvpages_append_axes if three else kv.kvpages_append
        assert call(pg.buf.t, pg.cfg, 0, n, 0, None, k, v, pg.slots, *more, None, None, 0.0, d, freq, None, None, None) == kv.KVP_OK
        torch.cuda.synchronize()
        images.append(pg.buf.t.cpu().numpy().copy())
    assert np.array_equal(*images)
