"""GPU tests of the page container: quantised writes with per-head norm and
rotation, reading back, and attention over pages joined with a base, against
the plain 64-bit forms in pageshelp.py.

Tolerances, from the roundings each output takes:
* held codes of unrotated rows: bit-exact (the formats' definition is in fp32
  operations that the plain form repeats);
* q_out, and bf16 keys: one bf16 rounding (2^-8 of the value) and fp32
  arithmetic on the pair (at most some 2^-19 of the row's largest pair norm);
* 8-bit keys: half a step of their scale (scale = max / 127, rounded to fp16:
  2^-11), the fp32 term, and one bf16 rounding on the way out;
* attention: one bf16 rounding of the result, weights rounded to 16 bits
  (2^-11 each: at most 2^-10 of sum p |v|); lse: fp32 sums of d products (2^-19
  of the largest sum of |q k|) and fp32 softmax sums.
"""
import math

import numpy as np
import pytest
import torch

import agent_shared_compressed_gb300 as kv
from agent_shared_compressed_gb300 import build as kvbuild
from agent_shared_compressed_gb300 import synth
import pageshelp as P
from kvhelp import CANARY_BYTES, Guarded

pytestmark = pytest.mark.gpu
FMTS = ["bf16", "k8v8", "k8v4"]


@pytest.fixture(scope="module", autouse=True)
def built():
    kvbuild.build()
    kv.load()


def _bf16(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.float32).to(torch.bfloat16)


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Pages:
    """A container full of NaN patterns, its table of scattered pages, and helpers."""

    def __init__(self, fmt, H, d, page, lens, L=1, layer=0, seed=0, spare=2, max_pages=None):
        self.fmt, self.H, self.d, self.P, self.lens, self.layer = fmt, H, d, page, list(lens), layer
        need = [(n + page - 1) // page for n in lens]
        self.max_pages = max_pages or max(1, max(need))
        self.n_pages = sum(need) + spare
        self.cfg = (L, H, d, page, self.n_pages, P.FORMATS[fmt])
        self.buf = Guarded(kv.kvpages_bytes(self.cfg), fill=0xFF)
        assert kv.kvpages_init(self.cfg, self.buf.t, self.buf.nbytes) == kv.KVP_OK
        rng = np.random.default_rng(seed)
        ids = rng.permutation(self.n_pages)
        self.table = np.full((len(lens), self.max_pages), -7, np.int32)  # entries past a sequence's end are never read
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at: at + n]
            at += n
        self.table_d = torch.from_numpy(self.table).cuda()
        self.lens_d = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.slots = torch.tensor([int(self.table[b, t // page]) * page + t % page for b, n in enumerate(lens)
                                   for t in range(n)], dtype=torch.int64, device="cuda")

    def append(self, k, v, slots=None, q=None, positions=None, q_norm=None, k_norm=None, eps=0.0, rot=0, freq=None,
               outs=True):
        n, nq = k.shape[0], 0 if q is None else q.shape[1]
        qo = Guarded(n * nq * self.d * 2) if nq else None
        ko, vo = (Guarded(n * self.H * self.d * 2) for _ in range(2)) if outs else (None, None)
        rc = kv.kvpages_append(self.buf.t, self.cfg, self.layer, n, nq, q, k, v, self.slots if slots is None else slots,
                               positions, q_norm, k_norm, eps, rot, freq, qo and qo.t, ko and ko.t, vo and vo.t)
        assert rc == kv.KVP_OK, kv.kvp_strerror(rc)
        torch.cuda.synchronize()
        assert self.buf.canary_ok() and all(g is None or g.canary_ok() for g in (qo, ko, vo))
        return (qo and _f64(qo.bf16((n, nq, self.d))), ko and _f64(ko.bf16((n, self.H, self.d))),
                vo and _f64(vo.bf16((n, self.H, self.d))))

    def read(self, max_tokens=None):
        T = max(1, max(self.lens)) if max_tokens is None else max_tokens
        shape = (len(self.lens), self.H, T, self.d)
        ko, vo = (Guarded(int(np.prod(shape)) * 2, fill=0x7F) for _ in range(2))
        rc = kv.kvpages_read(self.buf.t, self.cfg, self.layer, len(self.lens), self.table_d, self.max_pages, self.lens_d,
                             T, ko.t, vo.t)
        assert rc == kv.KVP_OK, kv.kvp_strerror(rc)
        torch.cuda.synchronize()
        assert ko.canary_ok() and vo.canary_ok()
        return _f64(ko.bf16(shape)), _f64(vo.bf16(shape))

    def attend(self, q, scale, base_out=None, base_lse=None, stream=None):
        B, m, nq, d = q.shape
        out, lse = Guarded(q.numel() * 2, fill=0x7F), Guarded(B * m * nq * 4, fill=0x7F)
        wsb = kv.kvpages_attend_workspace_bytes(self.cfg, B, m, nq)
        ws = Guarded(wsb, fill=0xFF)
        rc = kv.kvpages_attend(self.buf.t, self.cfg, self.layer, B, m, nq, q, scale, self.table_d, self.max_pages,
                               self.lens_d, base_out, base_lse, out.t, lse.t, ws.t, wsb, stream)
        assert rc == kv.KVP_OK, kv.kvp_strerror(rc)
        torch.cuda.synchronize()
        assert out.canary_ok() and lse.canary_ok() and ws.canary_ok() and self.buf.canary_ok()
        return _f64(out.bf16(q.shape)), lse.t.view(torch.float32).view(B, m, nq).cpu().numpy().astype(np.float64)

    def status(self):
        return kv.kvpages_status(self.buf.t)


def _kv(n, H, d, seed):
    k, v = synth.kv_layer(H, max(n, 1), d, torch.Generator().manual_seed(seed))
    return k.transpose(0, 1)[:n].contiguous().cuda(), v.transpose(0, 1)[:n].contiguous().cuda()


def _split(x, lens):
    cut = np.cumsum([0] + list(lens))
    return [x[cut[i]: cut[i + 1]] for i in range(len(lens))]


def _check_attend(out, lse, q, k, v, lens, scale, base=(None, None)):
    ref, ref_lse, mass, reach = P.attend(q, k, v, lens, scale, *base)
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mass + 1e-30
    err = np.abs(out - ref)
    assert np.all(err <= tol), "out: worst %.3g of its tolerance" % (err / tol).max()
    none = ~np.isfinite(ref_lse)
    assert np.array_equal(lse[none], ref_lse[none])
    tol = 2.0 ** -19 * (1 + np.abs(ref_lse[~none]) + reach[~none])
    err = np.abs(lse[~none] - ref_lse[~none])
    assert np.all(err <= tol), "lse: worst %.3g of its tolerance" % (err / tol).max()


# --- writing and reading back -------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H,d,page,lens", [(1, 128, 16, [1]), (3, 64, 16, [0, 37, 16, 1]), (8, 128, 64, [130, 15]),
                                           (2, 128, 1024, [1025]), (5, 64, 128, [200, 0])])
def test_write_and_read_back_exact(fmt, H, d, page, lens):
    """Unrotated rows: what the pages hold is the format's definition, bit for
    bit, from k_out / v_out and from reading back; rows past a length are zeros
    though the pages hold NaN patterns there."""
    pg = Pages(fmt, H, d, page, lens, L=2, layer=1, seed=d + H)
    k, v = _kv(sum(lens), H, d, 5)
    _, ko, vo = pg.append(k, v)
    hk, hv = P.to_bf16(P.held(_f64(k), fmt, False)), P.to_bf16(P.held(_f64(v), fmt, True))
    assert np.array_equal(ko, hk) and np.array_equal(vo, hv)
    T = max(lens) + 3
    rk, rv = pg.read(T)
    wk, wv = np.zeros_like(rk), np.zeros_like(rv)
    for b, (x, y) in enumerate(zip(_split(hk, lens), _split(hv, lens))):
        wk[b, :, :len(x)], wv[b, :, :len(y)] = x.transpose(1, 0, 2), y.transpose(1, 0, 2)
    assert np.array_equal(rk, wk) and np.array_equal(rv, wv)
    rk, rv = pg.read(max(1, max(lens) - 1))  # fewer rows than the longest sequence has
    assert np.array_equal(rk, wk[:, :, :rk.shape[2]]) and np.array_equal(rv, wv[:, :, :rv.shape[2]])
    assert pg.status() == kv.KVP_OK


@pytest.mark.parametrize("fmt", ["k8v8", "k8v4"])
def test_codes_at_borders(fmt):
    """Rows made of exact ties, zeros, constants, tiny and large values."""
    d, H = 128, 2
    rng = np.random.default_rng(1)
    rows = [np.zeros(d), np.full(d, 1.5), np.full(d, -2.0 ** -20), np.arange(d) * 1.0,
            np.where(np.arange(d) % 32 == 0, 127.0, (np.arange(d) % 32) + 0.5),       # s = 1: ties
            np.where(np.arange(d) % 32 == 0, 30.0, np.where(np.arange(d) % 32 == 1, 0.0, (np.arange(d) % 15) + 1.0)),
            1e-6 * rng.standard_normal(d), 3e4 * rng.standard_normal(d), 100 + 1e-2 * rng.standard_normal(d),
            np.where(np.arange(d) % 32 == 3, 1e4, 1e-3 * rng.standard_normal(d)), 2.0 ** -24 * np.ones(d)]
    x = _bf16(np.stack(rows)[:, None].repeat(H, 1)).cuda()
    x = torch.cat([x, -x, _bf16(rng.standard_normal((4000, H, d))).cuda()])
    pg = Pages(fmt, H, d, 64, [x.shape[0]])
    _, ko, vo = pg.append(x, x)
    assert np.array_equal(ko, P.to_bf16(P.held(_f64(x), fmt, False)))
    assert np.array_equal(vo, P.to_bf16(P.held(_f64(x), fmt, True)))
    # the large row has values below -65504: zero points past fp16
    assert pg.status() == (kv.KVP_ERR_RANGE if fmt == "k8v4" else kv.KVP_OK)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,nq,H,d,rot,norm", [(1, 32, 8, 128, 128, True), (15, 8, 8, 64, 64, False), (9, 5, 1, 128, 64, True),
                                               (70, 4, 2, 128, 128, False), (33, 6, 3, 64, 0, True),
                                               (1300, 2, 2, 64, 64, True)])
def test_norm_rotation_and_write(fmt, n, nq, H, d, rot, norm):
    """From the slices of a fused projection's output, at far positions."""
    g = torch.Generator().manual_seed(n + d)
    fused = torch.randn(n, nq + 2 * H, d, generator=g).to(torch.bfloat16).cuda()
    fused[:, :, 3] *= 20
    pos = torch.randint(0, 1 << 20, (n,), generator=g)
    pos[0], pos[-1] = (1 << 31) + 12345, 0
    freq = [500000.0 ** (-2.0 * i / rot) for i in range(rot // 2)] if rot else None
    w = [(0.5 + torch.rand(d, generator=g)).to(torch.bfloat16).cuda() if norm else None for _ in range(2)]
    pg = Pages(fmt, H, d, 32, [n])
    q, k, v = fused[:, :nq], fused[:, nq:nq + H], fused[:, nq + H:]
    qo, ko, vo = pg.append(k, v, q=q, positions=pos.cuda() if rot else None, q_norm=w[0], k_norm=w[1], eps=1e-6, rot=rot,
                           freq=freq)
    fw = [None if x is None else _f64(x) for x in w]
    rq, rk = (P.heads(_f64(x), y, 1e-6, pos.numpy(), freq, rot) for x, y in ((q, fw[0]), (k, fw[1])))
    fine = [2.0 ** -19 * np.abs(x).max(-1, keepdims=True) * math.sqrt(2) for x in (rq, rk)]
    assert np.all(np.abs(qo - rq) <= 2.0 ** -8 * np.abs(rq) + fine[0])
    if fmt == "bf16":
        step = 0.0
    else:
        top = np.abs(rk.reshape(n, H, -1, 32)).max(-1)
        step = (top / 127 * (0.5 + 2.0 ** -10)).repeat(32, -1)
    assert np.all(np.abs(ko - rk) <= step + 2.0 ** -8 * (np.abs(rk) + step) + fine[1])
    assert np.array_equal(vo, P.to_bf16(P.held(_f64(v), fmt, True)))
    hk, hv = pg.read()
    assert np.array_equal(hk[0].transpose(1, 0, 2), ko) and np.array_equal(hv[0].transpose(1, 0, 2), vo)
    assert pg.status() == kv.KVP_OK


def test_rows_by_head_and_in_place_queries():
    """[heads][tokens][dim] inputs; queries normed and turned in their own tensor."""
    H, nq, d, n = 2, 4, 128, 37
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(H, n, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(n, nq, d, generator=g).to(torch.bfloat16).cuda()
    freq = [0.01 * (i + 1) for i in range(64)]
    pos = torch.arange(n) + 7
    pg = Pages("bf16", H, d, 16, [n])
    rq, rk = (P.heads(_f64(x), None, 0.0, pos.numpy(), freq, 128) for x in (q, k.transpose(0, 1)))
    rc = kv.kvpages_append(pg.buf.t, pg.cfg, 0, n, nq, q, k.transpose(0, 1), v.transpose(0, 1), pg.slots, pos.cuda(), None,
                           None, 0.0, 128, freq, q, None, None)
    assert rc == kv.KVP_OK
    hk, hv = pg.read()
    assert np.all(np.abs(_f64(q) - rq) <= 2.0 ** -8 * np.abs(rq) + 2.0 ** -18 * np.abs(rq).max(-1, keepdims=True))
    assert np.all(np.abs(hk[0].transpose(1, 0, 2) - rk) <= 2.0 ** -8 * np.abs(rk) + 2.0 ** -18 * np.abs(rk).max(-1, keepdims=True))
    assert np.array_equal(hv[0], _f64(v))


def test_negative_slots_and_tokens_one_by_one():
    """A negative slot is not cached (its outputs are); a cache written token
    by token is the cache written at once, byte for byte."""
    H, d, n = 3, 128, 50
    k, v = _kv(n, H, d, 9)
    for fmt in FMTS:
        a, b = Pages(fmt, H, d, 16, [n], seed=4), Pages(fmt, H, d, 16, [n], seed=4)
        _, ka, va = a.append(k, v)
        for t in range(n):
            _, kt, vt = b.append(k[t:t + 1], v[t:t + 1], slots=b.slots[t:t + 1])
            assert np.array_equal(kt[0], ka[t]) and np.array_equal(vt[0], va[t])
        assert torch.equal(a.buf.t, b.buf.t)
        before = a.buf.t.clone()
        _, kt, vt = a.append(v, k, slots=torch.full((n,), -1, dtype=torch.int64, device="cuda"))
        assert torch.equal(before, a.buf.t) and np.array_equal(kt, P.to_bf16(P.held(_f64(v), fmt, False)))


def test_device_detected_errors():
    H, d = 2, 64
    k, v = _kv(20, H, d, 3)
    # a slot past the container: not written, reported; the others are
    pg = Pages("k8v8", H, d, 16, [20])
    slots = pg.slots.clone()
    slots[5] = pg.n_pages * 16
    slots[6] = 1 << 60
    pg.append(k, v, slots=slots)
    assert pg.status() == kv.KVP_ERR_PAGE
    hk = P.to_bf16(P.held(_f64(k), "k8v8", False))
    keep = [t for t in range(20) if t not in (5, 6)]
    assert np.array_equal(pg.read()[0][0].transpose(1, 0, 2)[keep], hk[keep])
    # Inf and NaN: coded as zeros where there are codes, kept in 16 bits
    bad_k, bad_v = k.clone(), v.clone()
    bad_k[3, 1, 7], bad_v[4, 0, 9] = float("inf"), float("nan")
    for fmt in FMTS:
        pg = Pages(fmt, H, d, 16, [20])
        _, ko, vo = pg.append(bad_k, bad_v)
        if fmt == "bf16":
            assert pg.status() == kv.KVP_OK and np.isinf(ko[3, 1, 7]) and np.isnan(vo[4, 0, 9])
            continue
        assert pg.status() == kv.KVP_ERR_NONFINITE
        zk, zv = bad_k.clone(), bad_v.clone()
        zk[3, 1, 7], zv[4, 0, 9] = 0.0, 0.0
        assert np.array_equal(ko, P.to_bf16(P.held(_f64(zk), fmt, False)))
        assert np.array_equal(vo, P.to_bf16(P.held(_f64(zv), fmt, True)))
    # a scale past fp16
    pg = Pages("k8v8", H, d, 16, [20])
    big = k.clone()
    big[0, 0, 0] = 1e7
    pg.append(big, v)
    assert pg.status() == kv.KVP_ERR_RANGE
    # not a container / another container
    pg = Pages("k8v8", H, d, 16, [20])
    other = (1, H, d, 16, pg.n_pages, P.FORMATS["k8v4"])
    q = torch.zeros(1, 1, H, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kv.kvpages_attend_workspace_bytes(other, 1, 1, H), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    assert kv.kvpages_attend(pg.buf.t, other, 0, 1, 1, H, q, 1.0, pg.table_d, pg.max_pages, pg.lens_d, None, None, out,
                             None, ws, ws.numel()) == kv.KVP_OK
    assert pg.status() == kv.KVP_ERR_HEADER
    assert kv.kvpages_status(torch.zeros(256, dtype=torch.uint8, device="cuda")) == kv.KVP_ERR_HEADER


def test_bad_pages_and_lengths():
    """Page ids outside the container and lengths past the table row: skipped
    (zeros when read), reported, and the other tokens unaffected."""
    H, d, page, lens = 2, 128, 16, [70, 33]
    for fmt in FMTS:
        k, v = _kv(sum(lens), H, d, 4)
        pg = Pages(fmt, H, d, page, lens)
        pg.append(k, v)
        hk, hv = P.held(_f64(k), fmt, False), P.held(_f64(v), fmt, True)
        q = torch.randn(2, 1, 4, d).to(torch.bfloat16).cuda()
        bad = pg.table.copy()
        bad[0, 2], bad[1, 1] = pg.n_pages, -1
        pg.table_d = torch.from_numpy(bad).cuda()
        out, lse = pg.attend(q, 0.1)
        keep = [[t for t in range(70) if t // 16 != 2], [t for t in range(33) if t // 16 != 1]]
        ks = [x[i] for x, i in zip(_split(hk, lens), keep)]
        vs = [x[i] for x, i in zip(_split(hv, lens), keep)]
        _check_attend(out, lse, _f64(q), ks, vs, [len(i) for i in keep], 0.1)
        assert pg.status() == kv.KVP_ERR_PAGE
        rk, _ = pg.read()
        assert not rk[0, :, 32:48].any() and np.array_equal(rk[0, :, 48:70].transpose(1, 0, 2), P.to_bf16(hk[48:70]))
        # a length past the table row is cut to it; a negative one is none
        pg = Pages(fmt, H, d, page, lens, max_pages=5)
        pg.append(k, v)
        pg.lens_d = torch.tensor([10 ** 6, -3], dtype=torch.int32, device="cuda")
        pg.table_d = torch.from_numpy(np.where(pg.table < 0, 0, pg.table)).cuda()
        out, lse = pg.attend(q, 0.1)
        assert pg.status() == kv.KVP_ERR_PAGE
        assert not out[1].any() and np.all(lse[1] == -np.inf)


# --- attention ------------------------------------------------------------------

ATTEND = [  # H, d, page, lens, m, query heads
    (1, 128, 16, [1], 1, 1),
    (8, 128, 16, [0, 1, 15, 16, 17, 31, 33], 1, 32),
    (2, 64, 32, [100, 0, 513, 64], 1, 8),
    (3, 128, 64, [700, 65], 1, 9),
    (4, 64, 128, [129, 128, 127], 1, 4),
    (2, 128, 16, [300, 2, 0, 5], 5, 8),     # a sequence shorter than its query tokens
    (1, 128, 32, [257, 40], 4, 16),         # 64 rows per KV head
    (2, 64, 16, [90, 3], 8, 6),
    (1, 64, 1024, [3000], 1, 12),
    (5, 128, 16, [40] * 21, 1, 5),
    (2, 128, 32, [333, 0, 20], 2, 8),       # 8 rows per KV head
    (1, 64, 16, [50, 1000], 1, 7),
    (2, 128, 64, [600, 3, 64], 1, 10),      # 5
    (1, 128, 16, [48, 47], 3, 2),           # 6
    (1, 64, 16, [10] * 40 + [0] * 3, 1, 4),  # more sequences than a warp has lanes
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", ATTEND)
def test_attend_matches_plain(fmt, case):
    H, d, page, lens, m, nq = case
    pg = Pages(fmt, H, d, page, lens, seed=len(lens))
    k, v = _kv(sum(lens), H, d, 11)
    pg.append(k, v, outs=False)
    ks = _split(P.held(_f64(k), fmt, False), lens)
    vs = _split(P.held(_f64(v), fmt, True), lens)
    g = torch.Generator().manual_seed(6)
    q = torch.randn(len(lens), m, nq, d, generator=g).to(torch.bfloat16)
    scale = 1.0 / math.sqrt(d)
    out, lse = pg.attend(q.cuda(), scale)
    _check_attend(out, lse, _f64(q), ks, vs, lens, scale)
    again = pg.attend(q.cuda(), scale)
    assert np.array_equal(out, again[0]) and np.array_equal(lse, again[1])
    bo, bl = torch.randn(q.shape, generator=g), torch.randn(q.shape[:3], generator=g) * 3
    bl[0, 0, 0] = -math.inf   # a base that saw nothing, with whatever its output holds
    bo[0, 0, 0] = 0.0
    out, lse = pg.attend(q.cuda(), scale, bo.cuda(), bl.cuda())
    _check_attend(out, lse, _f64(q), ks, vs, lens, scale, (bo.numpy().astype(np.float64), bl.numpy().astype(np.float64)))
    assert pg.status() == kv.KVP_OK


@pytest.mark.parametrize("fmt", FMTS)
def test_attend_extreme_scores_and_values(fmt):
    """One-hot and flat softmaxes, an attention sink with a tiny value, values
    from subnormal scales to large, zero keys, zero values, queries of any
    magnitude."""
    H, d, n = 1, 128, 200
    rng = np.random.default_rng(8)
    k = rng.standard_normal((n, H, d))
    v = rng.standard_normal((n, H, d))
    k[0] *= 8.0
    v[0] *= 1e-5                    # the sink
    v[50:60] *= 1e3
    v[60:70] = 0.0
    k[70:80] = 0.0
    v[80:90] *= 2e-5
    k, v = _bf16(k).cuda(), _bf16(v).cuda()
    pg = Pages(fmt, H, d, 16, [n])
    pg.append(k, v)
    hk, hv = [P.held(_f64(k), fmt, False)], [P.held(_f64(v), fmt, True)]
    q = np.concatenate([rng.standard_normal((1, 1, 4, d)), np.zeros((1, 1, 1, d)), _f64(k)[0][None, None],
                        1e-4 * rng.standard_normal((1, 1, 1, d)), 50.0 * rng.standard_normal((1, 1, 1, d))], 2)
    q = _bf16(q)
    for scale in (1.0 / math.sqrt(d), 2.0, 0.0, -0.3):
        out, lse = pg.attend(q.cuda(), scale)
        _check_attend(out, lse, _f64(q), hk, hv, [n], scale)
    # all values tiny; all values zero
    for f in (1e-6, 0.0):
        pg = Pages(fmt, H, d, 16, [n])
        w = _bf16(f * rng.standard_normal((n, H, d))).cuda()
        pg.append(k, w)
        out, lse = pg.attend(q.cuda(), 0.1)
        _check_attend(out, lse, _f64(q), hk, [P.held(_f64(w), fmt, True)], [n], 0.1)


@pytest.mark.parametrize("fmt", FMTS)
def test_attend_ignores_what_lies_past_the_lengths(fmt):
    """Written, then cut short: NaN, Inf and large tokens past the length, in
    the same page, change nothing; nor do other sequences' tokens."""
    H, d, n, cut = 2, 64, 77, 41
    k, v = _kv(n, H, d, 12)
    k2, v2 = k.clone(), v.clone()
    k2[cut:], v2[cut:] = float("nan"), float("inf")
    v2[cut + 1] = 3e38
    outs = []
    for a, b in ((k, v), (k2, v2)):
        pg = Pages(fmt, H, d, 32, [n])
        pg.append(a, b)
        pg.lens_d[0] = cut
        g = torch.Generator().manual_seed(1)
        q = torch.randn(1, 3, 4, d, generator=g).to(torch.bfloat16)
        outs.append(pg.attend(q.cuda(), 0.125))
    assert np.array_equal(outs[0][0], outs[1][0]) and np.array_equal(outs[0][1], outs[1][1])
    _check_attend(*outs[0], _f64(q), [P.held(_f64(k), fmt, False)[:cut]], [P.held(_f64(v), fmt, True)[:cut]], [cut], 0.125)


def test_shared_pages_and_other_layers():
    """Two sequences on the same first pages; three layers that do not mix."""
    H, d, page, lens = 2, 128, 16, [48, 48]
    for layer in (0, 2):
        pg = Pages("k8v8", H, d, page, lens, L=3, layer=layer)
        pg.table[1, :2] = pg.table[0, :2]
        pg.table_d = torch.from_numpy(pg.table).cuda()
        slots = torch.tensor([int(pg.table[b, t // page]) * page + t % page for b in range(2) for t in range(48)],
                             dtype=torch.int64, device="cuda")
        k, v = _kv(96, H, d, 13)
        k[48:80], v[48:80] = k[:32], v[:32]
        keep = torch.cat([torch.arange(48), torch.arange(80, 96)]).cuda()
        pg.append(k[keep].contiguous(), v[keep].contiguous(), slots=slots[keep])
        q = torch.randn(2, 1, 4, d).to(torch.bfloat16)
        out, lse = pg.attend(q.cuda(), 0.1)
        _check_attend(out, lse, _f64(q), _split(P.held(_f64(k), "k8v8", False), lens),
                      _split(P.held(_f64(v), "k8v8", True), lens), lens, 0.1)


def test_long_sequence_and_offsets_past_32_bits():
    """A container of over 4 GB whose sequence sits in its last pages, 20,000
    tokens over 1,250 pages."""
    H, d, page, n = 8, 128, 16, 20000
    n_pages = 128000
    cfg = (1, H, d, page, n_pages, kv.KVP_PAGES_K8V8)
    size = kv.kvpages_bytes(cfg)
    assert size > 1 << 32
    buf = torch.empty(size + CANARY_BYTES, dtype=torch.uint8, device="cuda")
    assert kv.kvpages_init(cfg, buf, size) == kv.KVP_OK
    ids = torch.arange(n_pages - 1, n_pages - 1 - n // page, -1, dtype=torch.int32)
    table = ids[None].cuda()
    slots = (ids.long()[:, None] * page + torch.arange(page)).flatten().cuda()
    k, v = _kv(n, H, d, 14)
    assert kv.kvpages_append(buf, cfg, 0, n, 0, None, k, v, slots, None, None, None, 0.0, 0, None, None, None, None) == 0
    q = torch.randn(1, 1, 16, d).to(torch.bfloat16)
    out, lse = torch.empty(1, 1, 16, d, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 1, 16, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    ws = torch.empty(kv.kvpages_attend_workspace_bytes(cfg, 1, 1, 16), dtype=torch.uint8, device="cuda")
    assert kv.kvpages_attend(buf, cfg, 0, 1, 1, 16, q.cuda(), 0.09, table, n // page, lens, None, None, out, lse, ws,
                             ws.numel()) == 0
    assert kv.kvpages_status(buf) == kv.KVP_OK
    _check_attend(_f64(out), lse.cpu().numpy().astype(np.float64), _f64(q), [P.held(_f64(k), "k8v8", False)],
                  [P.held(_f64(v), "k8v8", True)], [n], 0.09)


def test_streams_and_graphs():
    """Calls on another stream than the tensors' own, and a whole decode step
    captured once and replayed on new contents."""
    H, nq, d, lens = 2, 8, 128, [40, 3]
    k, v = _kv(sum(lens), H, d, 15)
    pg = Pages("k8v8", H, d, 16, lens)
    pg.append(k, v)
    ks, vs = _split(P.held(_f64(k), "k8v8", False), lens), _split(P.held(_f64(v), "k8v8", True), lens)
    q = torch.randn(2, 1, nq, d).to(torch.bfloat16).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = pg.attend(q, 0.1, stream=side)
    _check_attend(out, lse, _f64(q), ks, vs, lens, 0.1)
    # a step: append one token per sequence, attend over the cache with it
    new_q, new_k, new_v = (torch.zeros(2, h, d, dtype=torch.bfloat16, device="cuda") for h in (nq, H, H))
    last = torch.tensor([39, 42], device="cuda")
    slots, pos = pg.slots[last], torch.tensor([39, 2], device="cuda")
    freq = kv.binding._floats([0.5 ** i for i in range(64)])
    q_out = torch.empty_like(new_q)
    o, ls = torch.empty(2, 1, nq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 1, nq, device="cuda")
    ws = torch.empty(kv.kvpages_attend_workspace_bytes(pg.cfg, 2, 1, nq), dtype=torch.uint8, device="cuda")

    def step(st):
        assert kv.kvpages_append(pg.buf.t, pg.cfg, 0, 2, nq, new_q, new_k, new_v, slots, pos, None, None, 0.0, 128, freq,
                                 q_out, None, None, st) == 0
        assert kv.kvpages_attend(pg.buf.t, pg.cfg, 0, 2, 1, nq, q_out, 0.1, pg.table_d, pg.max_pages, pg.lens_d, None,
                                 None, o, ls, ws, ws.numel(), st) == 0

    with torch.cuda.stream(side):
        step(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(torch.cuda.current_stream())
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        a, b, c = (torch.randn(2, h, d, generator=g).to(torch.bfloat16) for h in (nq, H, H))
        new_q.copy_(a), new_k.copy_(b), new_v.copy_(c)
        graph.replay()
        torch.cuda.synchronize()
        w = np.array([0.5 ** i for i in range(64)], np.float32)
        rk = P.heads(_f64(b), None, 0, pos.cpu().numpy(), w, 128)
        held_k, held_v = pg.read()
        for i, n in enumerate(lens):
            s = np.abs(rk[i].reshape(H, 4, 32)).max(-1).repeat(32, -1) / 127
            assert np.all(np.abs(held_k[i, :, n - 1] - rk[i]) <= s * 0.51 + 2.0 ** -8 * (np.abs(rk[i]) + s))
            vs[i][n - 1] = P.held(_f64(c), "k8v8", True)[i]
            ks[i][n - 1] = P.held(rk, "k8v8", False)[i]
        rq = _f64(q_out)[:, None]
        ref, _, mass, reach = P.attend(rq, ks, vs, lens, 0.1)
        # the new key's codes may differ from the plain form's by a step where fp32 decides a tie
        far = 0.1 * np.abs(rq).sum(-1, keepdims=True) * np.abs(rk).max() / 127 * 2.0
        assert np.all(np.abs(_f64(o) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + far * 0.02) * mass)


def test_chained_calls_without_synchronisation():
    """Many steps back to back on one stream, the workspace reused by each."""
    H, nq, d, page, steps = 2, 4, 64, 16, 40
    pg = Pages("k8v4", H, d, page, [steps, steps])
    k, v = _kv(2 * steps, H, d, 16)
    outs, lses = [], []
    ws = torch.empty(kv.kvpages_attend_workspace_bytes(pg.cfg, 2, 1, nq), dtype=torch.uint8, device="cuda")
    q = torch.randn(steps, 2, 1, nq, d).to(torch.bfloat16).cuda()
    lens = [torch.tensor([t + 1, t + 1], dtype=torch.int32, device="cuda") for t in range(steps)]
    idx = [torch.tensor([t, steps + t], device="cuda") for t in range(steps)]
    ins = [(k[i].contiguous(), v[i].contiguous(), pg.slots[i].contiguous()) for i in idx]
    torch.cuda.synchronize()
    for t in range(steps):
        a, b, c = ins[t]
        assert kv.kvpages_append(pg.buf.t, pg.cfg, 0, 2, 0, None, a, b, c, None, None, None, 0.0, 0, None, None, None, None) == 0
        o, ls = torch.empty(2, 1, nq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 1, nq, device="cuda")
        assert kv.kvpages_attend(pg.buf.t, pg.cfg, 0, 2, 1, nq, q[t], 0.2, pg.table_d, pg.max_pages, lens[t], None, None,
                                 o, ls, ws, ws.numel()) == 0
        outs.append(o)
        lses.append(ls)
    torch.cuda.synchronize()
    hk, hv = P.held(_f64(k), "k8v4", False), P.held(_f64(v), "k8v4", True)
    for t in range(steps):
        ks, vs = [hk[:t + 1], hk[steps:steps + t + 1]], [hv[:t + 1], hv[steps:steps + t + 1]]
        _check_attend(_f64(outs[t]), lses[t].cpu().numpy().astype(np.float64), _f64(q[t]), ks, vs, [t + 1, t + 1], 0.2)


@pytest.mark.parametrize("fmt", FMTS)
def test_joined_with_the_pool(fmt):
    """Attention over the pool and over an agent's own pages, joined, is
    attention over both caches' tokens."""
    H, nq, d, T, lens = 2, 8, 128, 150, [33, 0, 90]
    shape = (1, H, d, T)
    ks_t, vs_t = synth.kv_layers(1, H, T, d, seed=3, device="cuda")
    pool = torch.empty(kv.kvpool_pool_bytes(shape), dtype=torch.uint8, device="cuda")
    pws = torch.empty(kv.kvpool_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    assert kv.kvpool_encode(shape, ks_t, vs_t, pool, pool.numel(), pws, pws.numel()) == 0
    pk, pv = (torch.empty(H, T, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kv.kvpool_decode_into(pool, shape, 0, 1, 1, [pk], [pv]) == 0
    q = torch.randn(3, 1, nq, d).to(torch.bfloat16).cuda()
    scale = 1.0 / math.sqrt(d)
    bo, bl = torch.empty(3, 1, nq, d, device="cuda"), torch.empty(3, 1, nq, device="cuda")
    aws = torch.empty(kv.kvpool_attend_workspace_bytes(shape, 3, nq), dtype=torch.uint8, device="cuda")
    assert kv.kvpool_attend(pool, shape, 0, 3, nq, q, scale, bo, bl, aws, aws.numel()) == 0
    pg = Pages(fmt, H, d, 16, lens)
    k, v = _kv(sum(lens), H, d, 17)
    pg.append(k, v)
    out, lse = pg.attend(q, scale, bo, bl)
    hk, hv = _split(P.held(_f64(k), fmt, False), lens), _split(P.held(_f64(v), fmt, True), lens)
    both_k = [np.concatenate([_f64(pk).transpose(1, 0, 2), x]) for x in hk]
    both_v = [np.concatenate([_f64(pv).transpose(1, 0, 2), x]) for x in hv]
    ref, ref_lse, mass, reach = P.attend(_f64(q), both_k, both_v, [T + n for n in lens], scale)
    # the decoded pool's bf16 keys and values stand for the pool's own: 2^-8 each
    assert np.all(np.abs(lse - ref_lse) <= 2.0 ** -8 * reach)
    assert np.all(np.abs(out - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -6 + 2.0 ** -7 * reach[..., None]) * mass)


def test_attend_wait_timeout_is_reported_and_context_survives():
    """With the next call limited to zero polls every warp gives up on its first
    block, lets its copies land and returns; the call after it is right."""
    H, d, lens = 4, 128, [900, 20]
    k, v = _kv(sum(lens), H, d, 18)
    pg = Pages("k8v8", H, d, 64, lens)
    pg.append(k, v)
    q = torch.randn(2, 1, 8, d).to(torch.bfloat16).cuda()
    assert kv.kvp_test_limit_next_pages_attend(0) == kv.KVP_OK
    pg.attend(q, 0.1)
    assert pg.status() == kv.KVP_ERR_TIMEOUT
    assert kv.kvpages_init(pg.cfg, pg.buf.t, pg.buf.nbytes) == kv.KVP_OK  # clears the error word; the pages stay
    out, lse = pg.attend(q, 0.1)
    assert pg.status() == kv.KVP_OK
    _check_attend(out, lse, _f64(q), _split(P.held(_f64(k), "k8v8", False), lens),
                  _split(P.held(_f64(v), "k8v8", True), lens), lens, 0.1)


@pytest.mark.parametrize("d", [64, 128])
def test_masked_draft_tokens_with_infinities(d):
    """16-bit pages: a drafted token whose value is Inf or NaN reaches the
    queries that see it and no others."""
    H, n, m = 2, 45, 4
    k, v = _kv(n, H, d, 19)
    v[n - 2, 0, 5], v[n - 1, 1, 9] = float("inf"), float("nan")
    pg = Pages("bf16", H, d, 16, [n])
    pg.append(k, v)
    q = torch.randn(1, m, 4, d).to(torch.bfloat16)
    out, lse = pg.attend(q.cuda(), 0.1)
    assert np.all(np.isfinite(out[0, :2])) and np.all(np.isfinite(lse))
    clean = v.clone()
    clean[n - 2:] = 0
    ref, _, mass, _ = P.attend(_f64(q), [_f64(k)], [_f64(clean)], [n], 0.1)
    assert np.all(np.abs(out[0, :2] - ref[0, :2]) <= 2.0 ** -8 * np.abs(ref[0, :2]) + 2.0 ** -10 * mass[0, :2])
    assert np.all(out[0, 2:, :2, 5] == np.inf) and np.all(np.isnan(out[0, 3, 2:, 9]))
    assert np.all(np.isfinite(out[0, 2, 2:]))
    # rows that see the Inf are right in their other dims
    keep = [i for i in range(d) if i != 5]
    full = v.clone()
    full[n - 2, 0, 5] = 0
    ref, _, mass, _ = P.attend(_f64(q), [_f64(k)], [_f64(full)], [n], 0.1)
    assert np.all(np.abs(out[0, 2:, :2][..., keep] - ref[0, 2:, :2][..., keep])
                  <= 2.0 ** -8 * np.abs(ref[0, 2:, :2][..., keep]) + 2.0 ** -10 * mass[0, 2:, :2][..., keep])


@pytest.mark.parametrize("fmt", FMTS)
def test_example_agent_decode(fmt):
    """The example's decode steps (pool, own pages, joined) against dense
    attention over the decoded caches.  Their bf16 keys move a score by up to
    2^-8 of sum |q k| (here below 0.4 where weights matter), their values and the
    output round to 2^-8."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "agent_decode.py")
    spec = importlib.util.spec_from_file_location("agent_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    worst, us = mod.run(agents=3, layers=2, heads=8, kv_heads=2, dim=128, pool_tokens=200, steps=20, fmt=fmt, check=True)
    assert worst < 0.02 and us > 0


@pytest.mark.parametrize("fmt,n,d", [("k8v8", 200, 128), ("k8v4", 700, 64), ("bf16", 4096, 64)])
def test_many_sequences(fmt, n, d):
    """More sequences than a thread block sums at once, up to the most of a call."""
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(0, 21 if n > 1000 else 60, n)]
    pg = Pages(fmt, 1, d, 16, lens, seed=1)
    k, v = _kv(sum(lens), 1, d, 20)
    pg.append(k, v, outs=False)
    q = torch.randn(n, 1, 2, d, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    out, lse = pg.attend(q.cuda(), 0.11)
    _check_attend(out, lse, _f64(q), _split(P.held(_f64(k), fmt, False), lens), _split(P.held(_f64(v), fmt, True), lens),
                  lens, 0.11)
    assert pg.status() == kv.KVP_OK


def test_norm_of_queries_or_keys_alone():
    H, nq, d, n = 2, 4, 128, 21
    g = torch.Generator().manual_seed(22)
    q, k = (torch.randn(n, h, d, generator=g).to(torch.bfloat16).cuda() for h in (nq, H))
    w = (0.5 + torch.rand(d, generator=g)).to(torch.bfloat16).cuda()
    for qn, kn in ((w, None), (None, w)):
        pg = Pages("bf16", H, d, 16, [n])
        qo, ko, _ = pg.append(k, k, q=q, q_norm=qn, k_norm=kn, eps=1e-6)
        for got, x, ww in ((qo, q, qn), (ko, k, kn)):
            ref = P.heads(_f64(x), None if ww is None else _f64(ww), 1e-6, None, None, 0)
            assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -10) if ww is not None else got == ref)


def test_calls_on_two_streams_at_once():
    """Two streams attend over one container at the same time, with workspaces
    and batches of their own; results are those of the calls one by one."""
    H, nq, d, lens = 4, 16, 128, [3000, 17, 900, 1]
    k, v = _kv(sum(lens), H, d, 23)
    pg = Pages("k8v8", H, d, 32, lens)
    pg.append(k, v, outs=False)
    g = torch.Generator().manual_seed(4)
    qs = [torch.randn(4, m, nq, d, generator=g).to(torch.bfloat16).cuda() for m in (1, 3)]
    alone = [pg.attend(q, 0.1) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    bufs = []
    for q in qs:
        wsb = kv.kvpages_attend_workspace_bytes(pg.cfg, 4, q.shape[1], nq)
        bufs.append([(torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")) for _ in range(20)]
                    + [torch.empty(wsb, dtype=torch.uint8, device="cuda")])
    torch.cuda.synchronize()
    for i in range(20):
        for q, st, b in zip(qs, streams, bufs):
            assert kv.kvpages_attend(pg.buf.t, pg.cfg, 0, 4, q.shape[1], nq, q, 0.1, pg.table_d, pg.max_pages, pg.lens_d,
                                     None, None, b[i][0], b[i][1], b[-1], b[-1].numel(), st) == 0
    torch.cuda.synchronize()
    for (out, lse), b in zip(alone, bufs):
        for o, ls in b[:-1]:
            assert np.array_equal(_f64(o), out) and np.array_equal(ls.cpu().numpy().astype(np.float64), lse)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", ATTEND)
def test_attend_with_a_roomy_table(fmt, case):
    """The same sequences with a table that could hold far more: the work is
    split another way, the results are those of the plain form all the same,
    empty rows and bases among them."""
    H, d, page, lens, m, nq = case
    pg = Pages(fmt, H, d, page, lens, seed=len(lens), max_pages=max(200, 65536 // page))
    k, v = _kv(sum(lens), H, d, 11)
    pg.append(k, v, outs=False)
    ks = _split(P.held(_f64(k), fmt, False), lens)
    vs = _split(P.held(_f64(v), fmt, True), lens)
    g = torch.Generator().manual_seed(6)
    q = torch.randn(len(lens), m, nq, d, generator=g).to(torch.bfloat16)
    out, lse = pg.attend(q.cuda(), 0.1)
    _check_attend(out, lse, _f64(q), ks, vs, lens, 0.1)
    bo, bl = torch.randn(q.shape, generator=g), torch.randn(q.shape[:3], generator=g) * 3
    out, lse = pg.attend(q.cuda(), 0.1, bo.cuda(), bl.cuda())
    _check_attend(out, lse, _f64(q), ks, vs, lens, 0.1, (bo.numpy().astype(np.float64), bl.numpy().astype(np.float64)))
    assert pg.status() == kv.KVP_OK


@pytest.mark.parametrize("roomy", [False, True])
def test_attend_wait_timeout_of_either_split(roomy):
    H, d, lens = 2, 64, [300, 20]
    k, v = _kv(sum(lens), H, d, 24)
    pg = Pages("k8v4", H, d, 64, lens, max_pages=4096 if roomy else None)
    pg.append(k, v)
    q = torch.randn(2, 1, 8, d).to(torch.bfloat16).cuda()
    assert kv.kvp_test_limit_next_pages_attend(0) == kv.KVP_OK
    pg.attend(q, 0.1)
    assert pg.status() == kv.KVP_ERR_TIMEOUT
    assert kv.kvpages_init(pg.cfg, pg.buf.t, pg.buf.nbytes) == kv.KVP_OK
    out, lse = pg.attend(q, 0.1)
    assert pg.status() == kv.KVP_OK
    _check_attend(out, lse, _f64(q), _split(P.held(_f64(k), "k8v4", False), lens),
                  _split(P.held(_f64(v), "k8v4", True), lens), lens, 0.1)


@pytest.mark.parametrize("fmt,d", [("bf16", 128), ("k8v8", 64), ("k8v8", 128), ("k8v4", 64), ("k8v4", 128)])
@pytest.mark.parametrize("n,m,nq", [(70, 1, 16), (140, 1, 4), (140, 3, 16), (220, 2, 8), (300, 1, 16), (600, 1, 8), (610, 1, 4)])
def test_attend_by_number_of_row_tiles(fmt, d, n, m, nq):
    """From few row tiles, which many warps share, to about one a warp, and more
    than the GPU has warps; ragged, with empty sequences and bases."""
    H = 4
    rng = np.random.default_rng(n + m)
    lens = [int(x) for x in rng.integers(0, 150, n)]
    lens[0], lens[1], lens[-1] = 150, 0, 1
    pg = Pages(fmt, H, d, 16, lens, seed=2)
    k, v = _kv(sum(lens), H, d, 25)
    pg.append(k, v, outs=False)
    ks = _split(P.held(_f64(k), fmt, False), lens)
    vs = _split(P.held(_f64(v), fmt, True), lens)
    g = torch.Generator().manual_seed(7)
    q = torch.randn(n, m, nq, d, generator=g).to(torch.bfloat16)
    out, lse = pg.attend(q.cuda(), 0.1)
    _check_attend(out, lse, _f64(q), ks, vs, lens, 0.1)
    bo, bl = torch.randn(q.shape, generator=g), torch.randn(q.shape[:3], generator=g) * 3
    out, lse = pg.attend(q.cuda(), 0.1, bo.cuda(), bl.cuda())
    _check_attend(out, lse, _f64(q), ks, vs, lens, 0.1, (bo.numpy().astype(np.float64), bl.numpy().astype(np.float64)))
    assert pg.status() == kv.KVP_OK


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("roomy", [False, True])
def test_attend_many_rows_of_many_sequences(fmt, roomy):
    """Several waves of row tiles (a short table), and several rows to a block of
    the merge (a roomy one)."""
    H, d, n, m, nq = 4, 64, 90, 16, 16
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 90, n)]
    lens[3] = 0
    pg = Pages(fmt, H, d, 16, lens, seed=3, max_pages=4096 if roomy else None)
    k, v = _kv(sum(lens), H, d, 26)
    pg.append(k, v, outs=False)
    g = torch.Generator().manual_seed(8)
    q = torch.randn(n, m, nq, d, generator=g).to(torch.bfloat16)
    bo, bl = torch.randn(q.shape, generator=g), torch.randn(q.shape[:3], generator=g) * 3
    out, lse = pg.attend(q.cuda(), 0.1, bo.cuda(), bl.cuda())
    _check_attend(out, lse, _f64(q), _split(P.held(_f64(k), fmt, False), lens), _split(P.held(_f64(v), fmt, True), lens),
                  lens, 0.1, (bo.numpy().astype(np.float64), bl.numpy().astype(np.float64)))
    assert pg.status() == kv.KVP_OK
