"""GPU tests of attention over pages where it can go wrong: bounded waits that
run out for some lanes only, joins in place, values that are Inf or
NaN, or near the end of bf16's range."""
import numpy as np
import pytest
import torch

import agent_shared_compressed_gb300 as kv
from agent_shared_compressed_gb300 import build as kvbuild
import pageshelp as P
import pagesweights as W
from test_gpu_pages import FMTS, Pages, _bf16, _check_attend, _f64, _kv, _split

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    kvbuild.build()
    kv.load()


# --- waits ------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lanes", [0x1, 0x80000000, 0x00010000, 0xAAAAAAAA])
@pytest.mark.parametrize("roomy", [False, True])
def test_wait_that_runs_out_for_some_lanes(fmt, lanes, roomy):
    """A wait that some lanes give up and others do not ends the warp's run as a
    whole, in either split of the work; the call after it is right."""
    H, d, lens = 4, 128, [900, 20, 0]
    k, v = _kv(sum(lens), H, d, 30)
    pg = Pages(fmt, H, d, 64, lens, max_pages=4096 if roomy else None)
    pg.append(k, v)
    q = torch.randn(3, 1, 8, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    assert kv.kvp_test_limit_next_pages_attend_lanes(0, lanes) == kv.KVP_OK
    pg.attend(q, 0.1)
    assert pg.status() == kv.KVP_ERR_TIMEOUT
    assert kv.kvpages_init(pg.cfg, pg.buf.t, pg.buf.nbytes) == kv.KVP_OK  # clears the error word; the pages stay
    out, lse = pg.attend(q, 0.1)
    assert pg.status() == kv.KVP_OK
    _check_attend(out, lse, _f64(q), _split(P.held(_f64(k), fmt, False), lens), _split(P.held(_f64(v), fmt, True), lens),
                  lens, 0.1)


# --- joins -------------------------------------------------------------------------

JOINS = [  # H, d, page, lens, m, query heads, table width: which part of the code ends a row
    (4, 128, 16, [40, 0, 7, 64], 1, 16, None),       # teams' merges and whole tiles, tiles of 4
    (4, 64, 16, [150, 3, 0], 3, 8, None),            # of 8
    (2, 128, 16, [90, 33], 8, 8, None),              # of 16
    (4, 128, 16, [4000, 0, 2500], 1, 16, 4096),      # cut from the list, joined
    (2, 64, 16, [3000, 900], 3, 8, 4096),
    (8, 128, 16, [20] * 300, 1, 32, 4096),           # many whole tiles of the list
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", JOINS)
def test_join_with_lse_in_place(fmt, case):
    """lse written over base_lse gives what another tensor for it gives, bit for bit."""
    H, d, page, lens, m, nq, width = case
    pg = Pages(fmt, H, d, page, lens, max_pages=width)
    k, v = _kv(sum(lens), H, d, 31)
    pg.append(k, v, outs=False)
    g = torch.Generator().manual_seed(2)
    q = torch.randn(len(lens), m, nq, d, generator=g).to(torch.bfloat16).cuda()
    bo, bl = torch.randn(q.shape, generator=g).cuda(), (torch.randn(q.shape[:3], generator=g) * 3).cuda()
    out, lse = pg.attend(q, 0.1, bo, bl)
    wsb = kv.kvpages_attend_workspace_bytes(pg.cfg, len(lens), m, nq)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    for _ in range(5):
        o, both = torch.empty_like(q), bl.clone()
        assert kv.kvpages_attend(pg.buf.t, pg.cfg, 0, len(lens), m, nq, q, 0.1, pg.table_d, pg.max_pages, pg.lens_d, bo,
                                 both, o, both, ws, wsb) == kv.KVP_OK
        torch.cuda.synchronize()
        assert np.array_equal(_f64(o), out) and np.array_equal(both.cpu().numpy().astype(np.float64), lse)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("width", [None, 4096])
def test_base_that_is_not_a_number(fmt, width):
    """A base whose lse is NaN gives NaN, also for queries that see no token of
    their own; one whose lse is -inf gives what there is, whatever it holds."""
    H, nq, d, lens = 2, 4, 64, [0, 40, 0, 40]
    pg = Pages(fmt, H, d, 16, lens, max_pages=width)
    k, v = _kv(sum(lens), H, d, 32)
    pg.append(k, v, outs=False)
    q = torch.randn(4, 1, nq, d, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    bo, bl = torch.full(q.shape, float("nan"), device="cuda"), torch.full(q.shape[:3], float("nan"), device="cuda")
    bl[2:] = -float("inf")
    out, lse = pg.attend(q, 0.1, bo, bl)
    alone = pg.attend(q, 0.1)
    assert np.all(np.isnan(lse[:2])) and np.all(np.isnan(out[:2]))
    assert np.array_equal(lse[2:], alone[1][2:]) and np.array_equal(out[2:], alone[0][2:])


# --- values that are Inf or NaN ------------------------------------------------------

def _check_with_infinities(out, lse, q, k, v, lens, scale, base=(None, None)):
    """A weight is positive, so an Inf value is an Inf of its dim for every query that
    sees its token (NaN beside an Inf of the other sign or a NaN); the other dims are
    those without it."""
    clean = [np.where(np.isfinite(x), x, 0.0) for x in v]
    ref, ref_lse, mass, reach = P.attend(q, k, clean, lens, scale, *base)
    B, m, nq, d = q.shape
    special = np.zeros((B, m, nq, d))
    for b in range(B):
        H = v[b].shape[1]
        for i in range(m):
            see = v[b][:max(0, lens[b] - (m - 1 - i))].repeat(nq // H, 1)
            up, down, nan = (f.any(0) for f in (see == np.inf, see == -np.inf, np.isnan(see)))
            special[b, i][up], special[b, i][down] = np.inf, -np.inf
            special[b, i][nan | (up & down)] = np.nan
    odd = special != 0
    assert np.array_equal(out[odd], special[odd], equal_nan=True)
    # bf16's half step, and 2^-17 of each weight, with fp32's 2^-19 of a score
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -17 + 2.0 ** -19 * (1 + reach[..., None])) * mass + 1e-30
    assert np.all(np.abs(out - ref)[~odd] <= tol[~odd])
    some = np.isfinite(ref_lse)
    assert np.all(np.abs(lse[some] - ref_lse[some]) <= 2.0 ** -19 * (1 + np.abs(ref_lse[some]) + reach[some]))


INFS = [  # H, d, page, lens, m, query heads, table width, places (sequence, token, head, dim, value)
    (1, 128, 16, [1], 1, 1, None, [(0, 0, 0, 5, 1)]),                        # its weight is 1: the second bf16 is 0
    (1, 64, 16, [1], 1, 1, None, [(0, 0, 0, 63, -1)]),
    (2, 128, 16, [45, 0, 200], 1, 8, None, [(0, 3, 0, 0, 1), (0, 44, 1, 9, -1), (2, 100, 1, 77, 1), (2, 30, 0, 7, 0)]),
    (2, 128, 16, [45, 0, 200], 1, 8, 4096, [(0, 3, 0, 0, 1), (0, 44, 1, 9, -1), (2, 100, 1, 77, 1), (2, 30, 0, 7, 0)]),
    (2, 64, 32, [130, 65], 4, 8, None, [(0, 129, 0, 1, 1), (0, 128, 0, 2, 1), (0, 5, 1, 3, -1), (1, 64, 0, 4, 0), (1, 0, 1, 5, 1)]),
    (2, 64, 32, [130, 65], 4, 8, 4096, [(0, 129, 0, 1, 1), (0, 128, 0, 2, 1), (0, 5, 1, 3, -1), (1, 64, 0, 4, 0), (1, 0, 1, 5, 1)]),
    (1, 128, 16, [70], 8, 4, None, [(0, 63, 0, 1, 1), (0, 64, 0, 1, -1), (0, 66, 0, 8, 1), (0, 9, 0, 100, 1)]),
    (1, 128, 64, [5000], 1, 4, None, [(0, 0, 0, 1, 1), (0, 2500, 0, 1, 1), (0, 2501, 0, 2, -1), (0, 4999, 0, 127, 1)]),
    (1, 128, 64, [5000], 1, 4, None, [(0, 17, 0, 1, 1), (0, 3333, 0, 1, -1)]),   # Inf - Inf, in different parts
]


@pytest.mark.parametrize("case", INFS)
def test_values_that_are_infinite(case):
    """16-bit pages keep Inf and NaN values: wherever the token lies, and however the
    work is split, they reach the queries that see it as they are, and no others."""
    H, d, page, lens, m, nq, width, places = case
    k, v = _kv(sum(lens), H, d, 33)
    start = np.cumsum([0] + lens)
    for b, t, h, x, sign in places:
        v[int(start[b]) + t, h, x] = sign * float("inf") if sign else float("nan")
    pg = Pages("bf16", H, d, page, lens, max_pages=width)
    pg.append(k, v, outs=False)
    g = torch.Generator().manual_seed(4)
    q = torch.randn(len(lens), m, nq, d, generator=g).to(torch.bfloat16)
    args = (_f64(q), _split(_f64(k), lens), _split(_f64(v), lens), lens, 0.1)
    _check_with_infinities(*pg.attend(q.cuda(), 0.1), *args)
    bo, bl = torch.randn(q.shape, generator=g), torch.randn(q.shape[:3], generator=g) * 3
    _check_with_infinities(*pg.attend(q.cuda(), 0.1, bo.cuda(), bl.cuda()), *args,
                           (bo.numpy().astype(np.float64), bl.numpy().astype(np.float64)))
    assert pg.status() == kv.KVP_OK


@pytest.mark.parametrize("width", [None, 4096])
@pytest.mark.parametrize("n,at", [(16, 3), (200, 3), (200, 190), (3000, 3), (3000, 2990)])
def test_infinite_value_of_a_weight_below_fp32(n, at, width):
    """The Inf token's weight is e^-300 of the others': positive all the same, before
    and after them, in their block and in another warp's part; and so is the whole
    sequence's share of a join with a base e^300 above it."""
    H, d = 1, 128
    rng = np.random.default_rng(9)
    k, v = 0.01 * rng.standard_normal((n, H, d)), rng.standard_normal((n, H, d))
    k[:, :, 0], k[at, :, 0], v[at, :, 6] = 10.0, -20.0, np.inf
    k, v = _bf16(k).cuda(), _bf16(v).cuda()
    q = torch.zeros(1, 1, 4, d, dtype=torch.bfloat16)
    q[..., 0] = 10.0
    pg = Pages("bf16", H, d, 16, [n], max_pages=width)
    pg.append(k, v, outs=False)
    args = (_f64(q), [_f64(k)], [_f64(v)], [n], 1.0)
    _check_with_infinities(*pg.attend(q.cuda(), 1.0), *args)
    bo, bl = torch.randn(q.shape, generator=torch.Generator().manual_seed(5)), torch.full(q.shape[:3], 400.0)
    _check_with_infinities(*pg.attend(q.cuda(), 1.0, bo.cuda(), bl.cuda()), *args,
                           (bo.numpy().astype(np.float64), bl.numpy().astype(np.float64)))


# --- values near the end of bf16's range ---------------------------------------------

@pytest.mark.parametrize("n,nq,m,width", [(1, 1, 1, None), (16, 4, 1, None), (300, 4, 1, None), (300, 8, 3, None),
                                          (300, 4, 1, 4096), (5000, 4, 1, None), (5000, 8, 2, None), (5000, 16, 4, None)])
@pytest.mark.parametrize("d", [64, 128])
def test_large_finite_values(n, nq, m, width, d):
    """Values up to the largest of bf16, scores that rise along the sequence by less
    and by more than the slack of the running maximum: a weighted mean of them is
    finite.  One dim holds them from the start, one only in the middle, the others
    ordinary values; the last token of the last case is Inf in one dim besides."""
    H = 1
    rng = np.random.default_rng(n + nq)
    k, v = 0.02 * rng.standard_normal((n, H, d)), rng.standard_normal((n, H, d))
    top = float(torch.finfo(torch.bfloat16).max)
    v[:, :, 3] = top
    v[n // 3:n // 2 + 1, :, 40] = -top * rng.random((n // 2 + 1 - n // 3, H))
    v[:, :, 41] = np.where(np.arange(n) % 2 == 0, top, -0.75 * top)[:, None]
    v[n // 2:, :, 50] = 2.0 ** 70
    if n == 5000 and m == 4:
        v[-1, :, 60], v[-1, :, 61] = np.inf, top
    for slope in (0.0, 4.0, 40.0):
        k[:, :, 0] = slope * np.arange(n)[:, None] / n
        kb, vb = _bf16(k).cuda(), _bf16(v).cuda()
        q = rng.standard_normal((1, m, nq, d))
        q[..., 0] = np.abs(q[..., 0]) + 0.5
        q = _bf16(q)
        pg = Pages("bf16", H, d, 16, [n], max_pages=width)
        pg.append(kb, vb, outs=False)
        out, lse = pg.attend(q.cuda(), 1.0)
        _check_with_infinities(out, lse, _f64(q), [_f64(kb)], [_f64(vb)], [n], 1.0)
        assert np.all(np.abs(out[..., 3] / top - 1) <= 2.0 ** -8)
        bo, bl = torch.randn(q.shape, generator=torch.Generator().manual_seed(n)) * 5e37, torch.full(q.shape[:3], 10.0)
        out, lse = pg.attend(q.cuda(), 1.0, bo.cuda(), bl.cuda())
        _check_with_infinities(out, lse, _f64(q), [_f64(kb)], [_f64(vb)], [n], 1.0,
                               (bo.numpy().astype(np.float64), bl.numpy().astype(np.float64)))


@pytest.mark.parametrize("n,nq,width", [(40, 4, None), (40, 8, 4096), (40, 16, None), (3000, 4, None), (3000, 8, None)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("first", [True, False])
def test_large_values_of_small_weights(n, nq, width, d, first):
    """Values up to the largest of bf16 whose weights are 2^-80 to 2^-110 of the
    others': what they contribute is of any size, beside others of ordinary size in
    their own dims and in the rest."""
    H = 1
    rng = np.random.default_rng(n + nq)
    k, v = 0.01 * rng.standard_normal((n, H, d)), rng.standard_normal((n, H, d))
    top = float(torch.finfo(torch.bfloat16).max)
    at = np.arange(4) + (1 if first else n - 7)
    k[:, :, 0] = 10.0
    k[at, 0, 0] = 10.0 - np.log(2.0) * np.array([80, 90, 100, 110]) / 8
    v[at, :, 5], v[at[::2], :, 9], v[at[1], :, 17] = top, -top, 2.0 ** 100
    v[at, :, 20 + np.arange(4)] = top
    k, v = _bf16(k).cuda(), _bf16(v).cuda()
    q = 0.1 * rng.standard_normal((1, 1, nq, d))
    q[..., 0] = 8.0
    q = _bf16(q)
    pg = Pages("bf16", H, d, 16, [n], max_pages=width)
    pg.append(k, v, outs=False)
    _check_with_infinities(*pg.attend(q.cuda(), 1.0), _f64(q), [_f64(k)], [_f64(v)], [n], 1.0)


def test_small_values_keep_their_bits():
    """Values of about 2^-100, where no large ones are: nothing is scaled."""
    H, d, n = 2, 128, 200
    k, v = _kv(n, H, d, 34)
    v = (v.float() * 2.0 ** -100).to(torch.bfloat16)
    pg = Pages("bf16", H, d, 16, [n])
    pg.append(k, v, outs=False)
    q = torch.randn(1, 1, 8, d, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    out, lse = pg.attend(q.cuda(), 0.1)
    ref, _, mass, reach = P.attend(_f64(q), [_f64(k)], [_f64(v)], [n], 0.1)
    # any of the n products may be zero where it is below fp32's normal range
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -17 + 2.0 ** -19 * (1 + reach[..., None])) * mass + n * 2.0 ** -126
    assert np.all(np.abs(out - ref) <= tol)


# --- long runs -----------------------------------------------------------------------

def _run_units(fmt, d, rows, lens, tiles):
    """Units of a warp's run and units whose addresses a warp holds at a time, as
    csrc/kvpages_attend.cu cuts the list (its PatShape and tile_units)."""
    quant, tile = fmt != "bf16", 4 if rows <= 4 else (8 if rows <= 8 else 16)
    warps = (8 if not quant or tile == 16 else 12) if d == 128 else (12 if tile == 16 else 16)
    blocks = 2 if quant and tile <= 8 else 1
    units = sum((n + 16 * blocks - 1 + 64) // (16 * blocks) for n in lens if n) * tiles
    n_warps = torch.cuda.get_device_properties(0).multi_processor_count * warps
    return (units + n_warps - 1) // n_warps, 32 // blocks


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,H,m,nq,lens", [
    (128, 8, 1, 32, [70000, 62016, 0, 65001, 64000]),    # tiles of 4
    (64, 8, 1, 16, [100000, 90001, 87, 95000, 99968]),
    (128, 4, 2, 16, [129000, 131072, 120001, 130000]),   # of 8
    (128, 4, 4, 16, [131072, 99000, 120001, 130000]),    # of 16
])
@pytest.mark.parametrize("bad", [False, True])
def test_runs_longer_than_the_address_window(fmt, d, H, m, nq, lens, bad):
    """A warp's lanes hold the addresses of its run's next 16 or 32 units and fetch
    more as it goes: runs of more than two such windows, in every format, with page
    ids outside the container beyond the first.  The table rows name the same few
    pages over and over, so the plain result needs each token once, by its count."""
    page, held = 16 if d == 64 else 64, 1024  # (pages of 16: a unit may lack either of its blocks)
    per, window = _run_units(fmt, d, m * nq // H, lens, H)
    assert per > 2 * window
    rng = np.random.default_rng(d + m)
    pg = Pages(fmt, H, d, page, [held])
    k, v = _kv(held, H, d, 35)
    pg.append(k, v, outs=False)
    hk, hv = P.held(_f64(k), fmt, False), P.held(_f64(v), fmt, True)
    width = max((n + page - 1) // page for n in lens)
    which = rng.integers(0, held // page, (len(lens), width))   # the held page that each entry names
    gone = np.zeros(which.shape, bool)
    if bad:
        gone = rng.random(which.shape) < 0.1
        gone[:, :2 * window * 32 // page] = False
    pg.table_d = torch.from_numpy(np.where(gone, pg.n_pages + rng.integers(0, 9, which.shape), pg.table[0][which]).astype(np.int32)).cuda()
    pg.max_pages, pg.lens_d = width, torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn(len(lens), m, nq, d, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16)
    out, lse = pg.attend(q.cuda(), 0.05)
    assert pg.status() == (kv.KVP_ERR_PAGE if bad else kv.KVP_OK)
    steps = 2 * per + 100  # additions to a sum: the run's blocks, the parts
    for b, n in enumerate(lens):
        for i in range(m):
            see = max(0, n - (m - 1 - i))
            t = np.arange(see)
            t = t[~gone[b, t // page]]
            count = np.bincount(which[b, t // page] * page + t % page, minlength=held).astype(np.float64)
            for j in range(nq):
                h, x = j // (nq // H), _f64(q[b, i, j])
                if not see:
                    assert not out[b, i, j].any() and lse[b, i, j] == -np.inf
                    continue
                s = 0.05 * (hk[:, h] @ x)
                reach = 0.05 * (np.abs(hk[:, h]) @ np.abs(x)).max()
                top = s[count > 0].max()
                e = np.where(count > 0, count * np.exp(s - top), 0.0)
                ref, mass = (e / e.sum()) @ hv[:, h], (e / e.sum()) @ np.abs(hv[:, h])
                fine = 2.0 ** -19 * (1 + reach) + steps * 2.0 ** -23
                assert np.all(np.abs(out[b, i, j] - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -17 + fine) * mass + 1e-30)
                ref_lse = top + np.log(e.sum())
                assert abs(lse[b, i, j] - ref_lse) <= fine + 2.0 ** -23 * abs(ref_lse)


# --- how exactly weights are held ------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("repeat", [1, 20, 400])
@pytest.mark.parametrize("rows", [1, 4, 7, 16, 20])
@pytest.mark.parametrize("width", [None, 4096])
def test_weights_are_held_to_2_17(fmt, d, repeat, rows, width):
    """Two terms that cancel leave the weights' roundings: 2^-17 of each, as the
    header says, where one bf16 or 11 bits would be several times the bound."""
    q, k, v, scale = W.sequence(fmt, d, repeat, rows, seed=rows)
    n = len(k)
    pg = Pages(fmt, 1, d, 16, [n], max_pages=width)
    pg.append(_bf16(k).cuda(), _bf16(v).cuda(), outs=False)
    q = q[None, None]
    hk, hv = P.held(k, fmt, False), P.held(v, fmt, True)
    out, _ = pg.attend(_bf16(q).cuda(), scale)
    ref, _, mass, reach = P.attend(q, [hk], [hv], [n], scale)
    tol = W.bound(ref, mass, reach[..., None], n // 16 + 20)
    assert np.all(np.abs(out - ref) <= tol), (np.abs(out - ref) / tol).max()
