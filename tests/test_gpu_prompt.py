"""GPU tests of attention of whole prompts against 64 bits.  Weights enter the value
product as bf16: 2^-8 of sum p |v| (their sum is taken before that)."""
import math

import numpy as np
import pytest
import torch

import agent_shared_compressed_gb300 as kv
from agent_shared_compressed_gb300 import build as kvbuild
import longhelp as Lg
from kvhelp import Guarded

pytestmark = pytest.mark.gpu
WEIGHTS = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def built():
    kvbuild.build()
    kv.load()


class Call:
    """Sequences of (new tokens, tokens behind them), their tensors, and one call."""

    def __init__(self, seqs, H, G, d, seed=0, layout="packed", gap=0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.seqs, self.H, self.nq, self.d = seqs, H, H * G, d
        self.q_first, self.k_first, n, t = [0], [], 0, gap
        for new, past in seqs:
            n += new
            self.q_first.append(n)
            self.k_first.append(t)
            t += new + past + gap
        self.n, self.t = n + gap, t
        q = Lg.bf16(spread * rng.standard_normal((self.n, self.nq, d))).cuda()
        k, v = (Lg.bf16(rng.standard_normal((self.t, H, d))).cuda() for _ in range(2))
        if layout == "fused":            # slices of one projection's rows, and a wider row for q
            x = torch.cat([k, v], 1)
            q = torch.cat([q, q.flip(0)], 1)[:, :self.nq]
            k, v = x[:, :H], x[:, H:]
        elif layout == "heads":
            q, k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
        self.q, self.k, self.v = q, k, v
        self.q_first_d, self.k_first_d, self.k_lens_d = (
            torch.tensor(x, dtype=torch.int32, device="cuda") for x in (self.q_first, self.k_first, [a + b for a, b in seqs]))
        self.error = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.shape = kv.PromptShape(len(seqs), self.n, self.t, self.nq, H, d)
        self.wsb = kv.kvprompt_workspace_bytes(self.shape)

    def launch(self, scale, window=0, sinks=0, base=(None, None), out=None, lse=None, ws=None, stream=None):
        rc = kv.kvprompt_attend(self.shape, self.q, self.k, self.v, self.q_first_d, self.k_first_d, self.k_lens_d, scale, window,
                                sinks, *base, out, lse, self.error, ws, self.wsb, stream)
        assert rc == kv.KVP_OK, kv.kvp_strerror(rc)

    def run(self, scale, window=0, sinks=0, base=(None, None)):
        out, lse = Guarded(max(16, self.n * self.nq * self.d * 2), fill=0x7F), Guarded(max(16, self.n * self.nq * 4), fill=0x7F)
        ws = Guarded(self.wsb, fill=0xFF)
        self.launch(scale, window, sinks, base, out.t, lse.t, ws.t)
        torch.cuda.synchronize()
        assert out.canary_ok() and lse.canary_ok() and ws.canary_ok()
        self.raw = out.t[:self.n * self.nq * self.d * 2].clone(), lse.t[:self.n * self.nq * 4].clone()
        return (Lg.f64(out.bf16((self.n, self.nq, self.d))),
                self.raw[1].view(torch.float32).view(self.n, self.nq).cpu().numpy().astype(np.float64))

    def check(self, out, lse, scale, window=0, sinks=0, base=(None, None), weights=WEIGHTS):
        q, k, v = Lg.f64(self.q), Lg.f64(self.k), Lg.f64(self.v)
        for b, (new, past) in enumerate(self.seqs):
            i, t = slice(self.q_first[b], self.q_first[b + 1]), slice(self.k_first[b], self.k_first[b] + new + past)
            ref, ref_lse, mass, reach = Lg.prompt(q[i], k[t], v[t], past, window, sinks, scale)
            if base[0] is not None:
                ref, ref_lse, mass = Lg.join(ref, ref_lse, mass, base[0][i].cpu().numpy().astype(np.float64),
                                             base[1][i].cpu().numpy().astype(np.float64))
            Lg.check(out[i], lse[i], ref, ref_lse, mass, reach, weights)
        # rows of no sequence stay as they were
        used = self.q_first[-1] * self.nq
        assert bool((self.raw[0][used * self.d * 2:] == 0x7F).all()) and bool((self.raw[1][used * 4:] == 0x7F).all())

    def both(self, scale=None, **more):
        scale = 1 / math.sqrt(self.d) if scale is None else scale
        out, lse = self.run(scale, **more)
        assert kv.kvprompt_status(self.error) == kv.KVP_OK
        self.check(out, lse, scale, **more)
        return out, lse

    def base(self, seed=0):
        rng = np.random.default_rng(seed)
        bo = torch.from_numpy(0.1 * rng.standard_normal((self.n, self.nq, self.d))).float().cuda()
        bl = torch.from_numpy(rng.uniform(2, 6, (self.n, self.nq))).float().cuda()
        bl[::3, 0] = -math.inf
        return bo, bl


SEQS = [[(1, 0)], [(1, 300)], [(17, 0), (1, 0), (0, 5), (0, 0), (33, 100)], [(128, 0)], [(129, 0), (127, 1)], [(256, 0)],
        [(257, 0), (3, 1000), (64, 64)], [(700, 0)], [(300, 513), (5, 0), (40, 2)]]


@pytest.mark.parametrize("seqs", SEQS, ids=str)
@pytest.mark.parametrize("H,G,d", [(1, 1, 128), (2, 4, 128), (2, 4, 64), (1, 3, 128), (3, 1, 64), (1, 8, 64), (1, 5, 128)])
def test_causal(seqs, H, G, d):
    Call(seqs, H, G, d, seed=len(seqs) + G).both()


@pytest.mark.parametrize("H,G,d", [(1, 128, 64), (1, 100, 128), (2, 33, 64), (1, 64, 128), (1, 127, 128)])
def test_many_heads_of_one(H, G, d):
    Call([(5, 0), (3, 140)], H, G, d).both()
    Call([(9, 300)], H, G, d).both(window=20, sinks=2)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 0), (64, 4), (128, 128), (129, 3), (100, 300), (300, 17), (2000, 5),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (31, 2 ** 31 - 1)])
@pytest.mark.parametrize("H,G,d", [(2, 4, 128), (3, 1, 64), (1, 3, 64)])
def test_windows(window, sinks, H, G, d):
    Call([(700, 0), (130, 333), (1, 600), (5, 0)], H, G, d, seed=window % 1000).both(window=window, sinks=sinks)


@pytest.mark.parametrize("window,sinks", [(40, 1), (40, 31), (40, 32), (40, 33), (300, 32), (256, 160)])
def test_first_tokens_apart_from_the_window(window, sinks):
    """First tokens that a narrow tile holds, and one more than that, behind a gap; scales of either
    sign and 0; few rows over many keys, which are split."""
    for d, scale in ((128, None), (64, -0.2), (128, 0.0)):
        Call([(140, 900), (1, 1100), (300, 0)], 2, 4, d, seed=sinks).both(scale=scale, window=window, sinks=sinks)
    Call([(3, 30000)], 1, 2, 64).both(window=9000 + window, sinks=sinks)


@pytest.mark.parametrize("layout", ["fused", "heads"])
@pytest.mark.parametrize("d", [64, 128])
def test_layouts(layout, d):
    Call([(200, 31), (3, 0), (77, 5)], 2, 4, d, layout=layout, gap=3).both(window=90, sinks=4)
    Call([(1, 0)], 1, 1, d, layout=layout).both()


def test_rows_of_no_sequence_and_joins():
    for d, window, sinks in ((128, 0, 0), (64, 50, 3)):
        c = Call([(140, 20), (0, 9), (31, 0)], 2, 4, d, gap=5)
        c.both(window=window, sinks=sinks, base=c.base())


def test_more_new_tokens_than_keys():
    """Places below 0: the first queries see nothing: zeros and -inf, or the base."""
    c = Call([(50, -20), (300, -299), (3, -3), (260, -130)], 1, 2, 128)
    c.both()
    c.both(base=c.base())
    c.both(window=10, sinks=1)


def test_no_keys_at_all():
    """Sequences without keys, and no rows of k and v (null pointers): zeros and -inf, or the base."""
    c = Call([(5, -5), (200, -200)], 1, 3, 64)
    assert c.t == 0
    c.k = c.v = kv.Rows(None, 64, 64)
    for base in ((None, None), c.base()):
        out, lse = c.run(0.1, 0, 0, base)
        assert kv.kvprompt_status(c.error) == kv.KVP_OK
        if base[0] is None:
            assert not out[:205].any() and np.all(lse[:205] == -np.inf)
        else:
            want = base[0].to(torch.bfloat16)
            want[base[1] == -math.inf] = 0
            assert np.array_equal(out, Lg.f64(want)) and np.array_equal(lse, base[1].cpu().numpy().astype(np.float64))


@pytest.mark.parametrize("seqs", [[(150, 10)], [(5, 20000)]])
def test_outputs_and_rows_anywhere(seqs):
    """Results on 16-byte boundaries only, the workspace too; sequences that do not begin with q's
    first row, and not in order in k; rows of none are left as they are."""
    c = Call(seqs, 2, 2, 128, gap=4)
    want, want_lse = c.run(0.1)
    n = c.n * c.nq * c.d
    for off in (8, 16):
        out = torch.full((n + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(c.wsb + 64, dtype=torch.uint8, device="cuda")
        lse = torch.full((c.n * c.nq + 4,), 3.0, device="cuda")
        c.launch(0.1, 0, 0, (None, None), out[off:off + n], lse[1:1 + c.n * c.nq], ws[16:16 + c.wsb])
        torch.cuda.synchronize()
        used = sum(a for a, _ in seqs) * c.nq
        assert np.array_equal(Lg.f64(out[off:off + used * c.d]), want.reshape(-1)[:used * c.d])
        assert np.array_equal(lse[1:1 + used].cpu().numpy().astype(np.float64), want_lse.reshape(-1)[:used])
        assert bool((out[:off] == 3).all()) and bool((out[off + used * c.d:] == 3).all()) and bool((lse[1 + used:] == 3).all())
    c = Call([(0, 0), (30, 40), (20, 0)], 1, 2, 64, gap=9)
    ref = c.run(0.1)
    q = c.q.clone()
    c.q[9:] = q[:-9]
    c.q_first_d += 9
    got = c.run(0.1)
    assert np.array_equal(got[0][9:59], ref[0][:50]) and np.array_equal(got[1][9:59], ref[1][:50])
    assert bool((c.raw[0][:9 * c.nq * c.d * 2] == 0x7F).all()) and bool((c.raw[1][:9 * c.nq * 4] == 0x7F).all())


def test_unseen_nonfinite_beside_the_first_tokens():
    """Inf in tokens that share a tile with the first ones: the queries whose window has left them
    behind do not meet it."""
    c = Call([(600, 0)], 1, 4, 128)
    clean = c.run(0.1, 64, 5)
    c.v[5:40] = math.inf
    out, lse = c.run(0.1, 64, 5)
    p = np.arange(600)
    sees = (p >= 5) & (p - 39 < 64)
    assert np.array_equal(~np.isfinite(out).all((1, 2)), sees)
    tol = 2.0 ** -6 * np.abs(clean[0]).max()
    assert np.all(np.abs(out[~sees] - clean[0][~sees]) <= tol) and np.all(np.abs(lse - clean[1]) <= 1e-4)


def test_sharp_negative_and_zero_scales():
    for scale in (3.0, -0.1, 0.0, 1e-30):
        Call([(150, 60)], 2, 2, 128, spread=2.0).both(scale=scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seqs", [[(200, 300)], [(16, 9000)]], ids=str)
def test_weights_and_results_are_rounded_once(d, seqs):
    """The mean square of the error is what one bf16 rounding of every weight and one of the result
    make: a weight's is even within half a step, 2^-8 / m of it for a significand m, whose 1 / m^2
    is 3 / (8 log 2) on average (m even by its logarithm); a result's has a twelfth of its step
    squared.  Both parts are about as large; a second rounding of either would make 1.5 of it."""
    c = Call(seqs, 2, 4, d, seed=d)
    scale = 1 / math.sqrt(d)
    out, _ = c.run(scale)
    q, k, v = Lg.f64(c.q), Lg.f64(c.k), Lg.f64(c.v)
    (new, past), = seqs
    see = np.arange(new + past)[None] <= past + np.arange(new)[:, None]
    off = expected = 0.0
    for j in range(c.nq):
        s = np.where(see, scale * (q[:new, j] @ k[:, j // 4].T), -np.inf)
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        ref = p @ v[:, j // 4]
        step = 2.0 ** (np.floor(np.log2(np.abs(ref))) - 7)
        off += ((out[:new, j] - ref) ** 2).sum()
        expected += (2.0 ** -16 / (8 * math.log(2)) * (p ** 2 @ v[:, j // 4] ** 2) + step ** 2 / 12).sum()
    assert off <= 1.25 * expected, off / expected


def test_scores_that_rise_and_fall():
    """The running maximum raised in every tile, by hundreds; and falling ones."""
    for order in (1, -1):
        c = Call([(300, 700)], 1, 2, 64)
        size = torch.linspace(0.05, 6.0, c.t, device="cuda")[::1]
        c.q[:] = c.q.abs()
        c.k.copy_((c.k.abs().float() * (size if order == 1 else size.flip(0))[:, None, None]).to(torch.bfloat16))
        c.both(scale=0.5)


def _exact_scores(c, size, seed=0):
    """Queries and keys whose products and sums fp32 holds exactly: `size` times small whole numbers."""
    rng = np.random.default_rng(seed)
    c.q.copy_(Lg.bf16(size * rng.integers(-1, 2, c.q.shape)))
    c.k.copy_(Lg.bf16(size * rng.integers(-3, 4, c.k.shape)))


@pytest.mark.parametrize("size", [2.0 ** x for x in (4, 8, 9, 10, 13, 15, 17, 30, 59)])
def test_large_scores(size):
    """Scores up to 2^123: sums of products are exact, and keys that differ do so by a twelfth of
    size^2 or more: a row's result is the mean of the values whose keys score most."""
    for seqs, H, G, d, window, sinks in (([(300, 40), (140, 900)], 2, 4, 128, 0, 0), ([(300, 0), (5, 700)], 3, 1, 64, 70, 3),
                                         ([(200, 513)], 1, 3, 128, 300, 17), ([(3, 30000)], 1, 2, 64, 0, 0)):
        c = Call(seqs, H, G, d, seed=d + window)
        _exact_scores(c, size)
        for scale, base in ((1 / math.sqrt(d), False), (-1 / math.sqrt(d), True)):
            bo, bl = c.base() if base else (None, None)
            out, lse = c.run(scale, window, sinks, (bo, bl))
            assert kv.kvprompt_status(c.error) == kv.KVP_OK
            q, k, v = Lg.f64(c.q), Lg.f64(c.k), Lg.f64(c.v)
            for b, (new, past) in enumerate(seqs):
                i, t = slice(c.q_first[b], c.q_first[b + 1]), slice(c.k_first[b], c.k_first[b] + new + past)
                ref, ref_lse, mass, reach = Lg.prompt(q[i], k[t], v[t], past, window, sinks, scale)
                if base:
                    ref, ref_lse, mass = Lg.join(ref, ref_lse, mass, bo[i].cpu().numpy().astype(np.float64),
                                                 bl[i].cpu().numpy().astype(np.float64))
                # (what the scale's and the product's roundings make is the same for keys of one score;
                # of the lse they are 2^-22)
                Lg.check(out[i], lse[i], ref, ref_lse, mass, 0 * reach, WEIGHTS)


@pytest.mark.parametrize("size", [1e3, 4e4, 1e5, 1e9])
def test_large_random_scores(size):
    """Normal queries and keys of any size: fp32 does not say which of two keys scores more, but
    weights still make up a mean: of ones it is one (the weights' rounding and the result's, 2^-8
    each), of bf16's largest finite."""
    for seqs, H, G, d, window, sinks in (([(300, 40), (140, 900)], 2, 4, 128, 0, 0), ([(300, 0), (5, 700)], 3, 1, 64, 70, 3),
                                         ([(3, 30000)], 1, 2, 64, 0, 0)):
        c = Call(seqs, H, G, d, seed=d)
        c.q.mul_(size)
        c.k.mul_(size)
        c.v.fill_(1.0)
        out, lse = c.run(1 / math.sqrt(d), window, sinks)
        assert np.all(np.abs(out - 1.0) <= 2.0 ** -7)
        c.check(out, lse, 1 / math.sqrt(d), window, sinks)                     # the lse
        c.v.fill_(3.3895313892515355e38)
        out, _ = c.run(1 / math.sqrt(d), window, sinks)
        assert np.all(np.isfinite(out)) and np.all(out >= 3.3e38)


def test_shared_rows():
    """Two sequences over the same keys (a shared prefix), one over a part of them."""
    c = Call([(40, 100), (40, 100), (10, 20)], 2, 2, 128)
    c.k_first = [0, 0, 37]
    c.k_first_d.copy_(torch.tensor(c.k_first, dtype=torch.int32))
    c.both()
    c.both(window=33, sinks=5)


@pytest.mark.parametrize("d", [64, 128])
def test_unseen_nonfinite(d):
    """Inf and NaN in keys and values that a query does not see have no part: behind the
    last key, between sequences, in the window's gap, and later tokens of the prompt's own
    tiles; what is seen makes its dim Inf or NaN, for the queries that see it alone."""
    for window, sinks in ((0, 0), (70, 3)):
        c = Call([(300, 40), (129, 0)], 2, 4, d, gap=7)
        c.both(window=window, sinks=sinks)
        clean = c.run(0.1, window, sinks)
        inside = torch.zeros(c.t, dtype=torch.bool, device="cuda")
        for b, (new, past) in enumerate(c.seqs):
            inside[c.k_first[b]:c.k_first[b] + new + past] = True
        for x in (c.k, c.v):
            x[~inside] = math.nan
        got = c.run(0.1, window, sinks)
        assert np.array_equal(got[0], clean[0], equal_nan=True) and np.array_equal(got[1], clean[1], equal_nan=True)
        at, dim = 150, 5                       # token 150 of the first sequence: query 110
        c.v[c.k_first[0] + at, 1, dim] = math.inf
        c.v[c.k_first[0] + at, 0, dim + 1] = math.nan
        out, lse = c.run(0.1, window, sinks)
        q = np.arange(300)
        sees = (40 + q >= at) & ((40 + q - at < window) if window else True)
        assert np.array_equal(~np.isfinite(out[:300, 4:, dim]), np.repeat(sees[:, None], 4, 1))
        assert np.array_equal(~np.isfinite(out[:300, :4, dim + 1]), np.repeat(sees[:, None], 4, 1))
        rest = np.delete(out[:300], [dim, dim + 1], -1)
        tol = 2.0 ** -6 * np.abs(clean[0][:300]).max()
        assert np.all(np.abs(rest - np.delete(clean[0][:300], [dim, dim + 1], -1)) <= tol)
        assert np.all(np.abs(out[:300][~sees] - clean[0][:300][~sees]) <= tol)
        assert np.all(np.abs(lse[:300] - clean[1][:300]) <= 1e-4) and np.array_equal(out[300:429], clean[0][300:429])
        # a key that is NaN takes the rows that see it, and no others
        c.v.nan_to_num_(0.0, 0.0, 0.0)
        c.k[c.k_first[0] + at] = math.nan
        out, lse = c.run(0.1, window, sinks)
        assert np.array_equal(np.isnan(out[:300]).all((1, 2)), sees) and np.array_equal(np.isnan(out[:300]).any((1, 2)), sees)
        assert np.array_equal(np.isnan(lse[:300]).any(1), sees)


@pytest.mark.parametrize("d,times", [(64, 80), (128, 80), (128, 1)])
def test_unseen_nonfinite_over_many_keys(d, times):
    """A block that meets Inf or NaN has no more to do for its sequence being long: no other
    warp's wait runs out (sequences of 40256 keys, as many as fill the GPU, and one, which is
    split).  What does not see them is what it was, bit for bit."""
    c = Call([(256, 40000)], 2, 1, d)
    c.seqs, c.n = c.seqs * times, 256 * times
    c.q = c.q.repeat(times, 1, 1)
    c.q_first_d = torch.arange(0, c.n + 1, 256, dtype=torch.int32, device="cuda")
    c.k_first_d, c.k_lens_d = (torch.full((times,), x, dtype=torch.int32, device="cuda") for x in (0, 40256))
    c.shape = kv.PromptShape(times, c.n, c.t, c.nq, c.H, d)
    c.wsb = kv.kvprompt_workspace_bytes(c.shape)
    at = [(0, 40100, 3, math.inf), (0, 40100, d - 1, -math.inf), (1, 40255, 7, math.nan), (1, 40000, 33, math.inf)]
    for window, sinks, scale in ((0, 0, 0.1), (30000, 9, 0.1), (0, 0, 0.0)):
        clean = c.run(scale, window, sinks)
        was = c.v.clone()
        for h, t, e, x in at:
            c.v[t, h, e] = x
        out, lse = c.run(scale, window, sinks)
        c.v = was
        assert kv.kvprompt_status(c.error) == kv.KVP_OK
        want = clean[0].reshape(times, 256, 2, d)
        got = out.reshape(want.shape)
        for h, t, e, x in at:
            sees = 40000 + np.arange(256) >= t
            assert np.array_equal(got[:, :, h, e] == x if math.isinf(x) else np.isnan(got[:, :, h, e]), np.broadcast_to(sees, (times, 256)))
            want[:, sees, h, e] = got[:, sees, h, e]
        assert np.array_equal(got, want, equal_nan=True) and np.array_equal(lse, clean[1])


@pytest.mark.parametrize("d", [64, 128])
def test_values_up_to_the_largest(d):
    """Finite values give finite results up to bf16's largest, whatever the sums before
    the division would be."""
    c = Call([(200, 900)], 1, 2, d)
    c.v.fill_(3.3895313892515355e38)
    c.v[::2, :, ::2] *= -1
    out, lse = c.run(0.01)
    assert np.all(np.isfinite(out)) and np.all(np.isfinite(lse))
    assert np.all(np.abs(out[:, :, 1::2]) >= 3.3e38)


def test_ranges_outside_the_tensors():
    """A sequence whose numbers point outside is skipped and reported; the others are
    as they were."""
    good = Call([(40, 10), (20, 0), (30, 5)], 2, 2, 64)
    out, lse = good.run(0.1)
    for what, at, value in (("k_lens_d", 1, 1000), ("k_lens_d", 1, -1), ("k_first_d", 1, -1), ("k_first_d", 1, good.t - 5),
                            ("k_first_d", 1, 2 ** 31 - 1), ("k_lens_d", 1, 2 ** 31 - 1)):
        c = Call([(40, 10), (20, 0), (30, 5)], 2, 2, 64)
        getattr(c, what)[at] = value
        o, l = c.run(0.1)
        assert kv.kvprompt_status(c.error) == kv.KVP_ERR_PAGE
        for i in (slice(0, 40), slice(60, 90)):
            assert np.array_equal(o[i], out[i]) and np.array_equal(l[i], lse[i])
        assert bool((c.raw[1].view(torch.int32).view(-1, 4)[40:60] == 0x7F7F7F7F).all())
    c = Call([(40, 10), (20, 0), (30, 5)], 2, 2, 64)
    c.q_first_d[3] = 91                                                 # past q's rows
    c.run(0.1)
    assert kv.kvprompt_status(c.error) == kv.KVP_ERR_PAGE
    c = Call([(40, 10)], 2, 2, 64)
    c.q_first_d[0] = 50                                                 # decreasing
    c.run(0.1)
    assert kv.kvprompt_status(c.error) in (kv.KVP_OK, kv.KVP_ERR_PAGE)


def test_numbers_of_new_tokens_that_decrease():
    """They are reported wherever they are, and nothing outside the calls' rows is written (a
    sequence alone: nothing at all)."""
    c = Call([(40, 10)], 2, 2, 64)
    c.q_first_d[0] = 50
    c.run(0.1)
    assert kv.kvprompt_status(c.error) == kv.KVP_ERR_PAGE
    assert bool((c.raw[0] == 0x7F).all()) and bool((c.raw[1] == 0x7F).all())
    for seqs, at, value in (([(500, 0), (20, 0), (80, 0)], 2, 100), ([(500, 0), (20, 0), (80, 0)], 1, 590),
                            ([(3, 20000), (2, 0), (700, 0), (6, 0)], 3, 4), ([(7, 2)] * 700, 350, 3), ([(7, 2)] * 700, 699, 0),
                            ([(7, 2)] * 700, 0, 4000), ([(7, 2)] * 700, 40, 4899)):
        c = Call(seqs, 2, 2, 64, gap=3)
        c.q_first_d[at] = value
        c.run(0.1)
        assert kv.kvprompt_status(c.error) == kv.KVP_ERR_PAGE, (at, value)
        used = sum(a for a, _ in seqs) * c.nq
        assert bool((c.raw[0][used * c.d * 2:] == 0x7F).all()) and bool((c.raw[1][used * 4:] == 0x7F).all())


def test_many_sequences():
    """More sequences than tiles, empty ones among them."""
    rng = np.random.default_rng(0)
    seqs = [(int(a), int(b)) for a, b in zip(rng.integers(0, 7, 700), rng.integers(0, 40, 700))]
    Call(seqs, 2, 2, 64).both(window=9, sinks=2)


def test_hardly_any_work_among_many_numbers():
    """65536 sequences of 1024 heads, all but the first and the last empty: the blocks look at 67
    million numbers, longer than a wait may be, before the first one's."""
    H, d, B = 1024, 64, kv.KVP_PROMPT_MAX_SEQS
    c = Call([(3, 6), (2, 0)], H, 1, d)
    want = c.run(0.1)
    c.q_first_d = torch.full((B + 1,), 3, dtype=torch.int32, device="cuda")
    c.q_first_d[0], c.q_first_d[B] = 0, 5
    c.k_first_d, c.k_lens_d = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.full((B,), 9, dtype=torch.int32, device="cuda")
    c.k_first_d[B - 1], c.k_lens_d[B - 1] = 9, 2
    c.shape = kv.PromptShape(B, c.n, c.t, c.nq, H, d)
    c.wsb = kv.kvprompt_workspace_bytes(c.shape)
    got = c.run(0.1)
    assert kv.kvprompt_status(c.error) == kv.KVP_OK
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_few_rows_over_many_keys():
    for H, G, d, seqs in ((2, 4, 128, [(5, 20000)]), (1, 1, 64, [(1, 33333), (2, 70)]), (8, 4, 128, [(64, 5000)])):
        c = Call(seqs, H, G, d)
        c.both()
        c.both(base=c.base(), window=9000, sinks=200)


def test_same_results_every_time_and_on_two_streams():
    """Two calls at once, each with a workspace of its own; results do not depend on
    timing."""
    c = Call([(300, 3000), (40, 0)], 2, 4, 128)
    want = c.run(0.1)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    torch.cuda.synchronize()
    for i in range(6):
        out, lse = torch.empty(c.n, c.nq, c.d, dtype=torch.bfloat16, device="cuda"), torch.empty(c.n, c.nq, device="cuda")
        got.append((out, lse, torch.empty(c.wsb, dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    for i, (out, lse, ws) in enumerate(got):
        c.launch(0.1, 0, 0, (None, None), out, lse, ws, streams[i % 2])
    torch.cuda.synchronize()
    for out, lse, _ in got:
        assert np.array_equal(Lg.f64(out), want[0]) and np.array_equal(lse.cpu().numpy().astype(np.float64), want[1])


def test_in_graphs_as_lengths_change():
    """Captured once and replayed with other lengths; two graphs that run one after the
    other may share a workspace."""
    c = Call([(200, 100), (60, 0)], 2, 2, 128)
    graphs = []
    ws = torch.empty(c.wsb, dtype=torch.uint8, device="cuda")
    for window, sinks in ((0, 0), (50, 3)):
        out, lse = Guarded(c.n * c.nq * c.d * 2, fill=0x7F), Guarded(c.n * c.nq * 4, fill=0x7F)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            c.launch(0.1, window, sinks, (None, None), out.t, lse.t, ws, torch.cuda.current_stream())
        graphs.append((g, window, sinks, out, lse))
    for seqs in ([(200, 100), (60, 0)], [(1, 3), (2, 0)], [(0, 0), (260, 40)], [(130, 7), (129, 1)]):
        c.seqs = seqs
        c.q_first = [0, seqs[0][0], seqs[0][0] + seqs[1][0]]
        c.k_first = [0, sum(seqs[0])]
        for x, y in ((c.q_first_d, c.q_first), (c.k_first_d, c.k_first), (c.k_lens_d, [sum(s) for s in seqs])):
            x.copy_(torch.tensor(y, dtype=torch.int32))
        for g, window, sinks, out, lse in graphs:
            out.t.fill_(0x7F)
            lse.t.fill_(0x7F)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            c.raw = out.t[:c.n * c.nq * c.d * 2].clone(), lse.t[:c.n * c.nq * 4].clone()
            c.check(Lg.f64(out.bf16((c.n, c.nq, c.d))),
                    c.raw[1].view(torch.float32).view(c.n, c.nq).cpu().numpy().astype(np.float64), 0.1, window, sinks)


def test_lse_in_place_and_without():
    c = Call([(100, 30)], 2, 2, 128)
    bo, bl = c.base()
    want = c.both(base=(bo, bl))
    out = torch.empty(c.n, c.nq, c.d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(c.wsb, dtype=torch.uint8, device="cuda")
    scale = 1 / math.sqrt(128)
    c.launch(scale, 0, 0, (bo, bl), out, None, ws)
    torch.cuda.synchronize()
    assert np.array_equal(Lg.f64(out), want[0])
    c.launch(scale, 0, 0, (bo, bl), out, bl, ws)
    torch.cuda.synchronize()
    assert np.array_equal(Lg.f64(out), want[0]) and np.array_equal(bl.cpu().numpy().astype(np.float64), want[1])


def test_rows_past_two_gigabytes():
    """Keys and values whose offsets pass 32 bits: a sequence at the end of 2^25 rows."""
    H, d, rows = 1, 128, (1 << 25) + 500
    c = Call([(70, 300)], H, 2, d)
    k = torch.zeros(rows, H, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    at = rows - c.t
    k[at:], v[at:] = c.k, c.v
    want = c.run(0.1)
    c.k, c.v = k, v
    c.k_first_d.fill_(at)
    c.shape = kv.PromptShape(1, c.n, rows, c.nq, H, d)
    c.wsb = kv.kvprompt_workspace_bytes(c.shape)
    got = c.run(0.1)
    assert np.allclose(got[0], want[0], rtol=2.0 ** -7, atol=2.0 ** -10) and np.allclose(got[1], want[1], atol=1e-5)


def test_wait_that_runs_out_is_reported():
    """The next call polls for no copy at all: it gives up, reports it, and leaves the
    context usable."""
    for splits in (False, True):
        c = Call([(5, 20000)] if splits else [(300, 40), (3, 0)], 2, 2, 128)
        want = c.run(0.1)
        kv.kvp_test_limit_next_prompt(0)
        c.run(0.1)
        assert kv.kvprompt_status(c.error) == kv.KVP_ERR_TIMEOUT
        c.error.zero_()
        got = c.run(0.1)
        assert kv.kvprompt_status(c.error) == kv.KVP_OK
        assert np.array_equal(got[0], want[0], equal_nan=True) and np.array_equal(got[1], want[1], equal_nan=True)
