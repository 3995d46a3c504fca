"""Plain 64-bit forms of the operators for agents that live long: a window with
first tokens, caches in 4 bits, positions of several axes, whole prompts.  Shares
no code with the library."""
import numpy as np
import torch

import agent_shared_compressed_gb300 as kv
import pageshelp as P
from kvhelp import Guarded

FORMATS = dict(P.FORMATS, k4v4=4)


def bf16(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.float32).to(torch.bfloat16)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def held(x, fmt, values):
    """What a page of the format holds for fp32 x."""
    return P.held4(x) if fmt == "k4v4" else P.held(x, fmt, values)


def held8(x):
    """What 8-bit codes hold for fp32 x, scales beyond fp16 held at its largest too."""
    g = np.asarray(x, np.float32).reshape(*np.shape(x)[:-1], -1, 32)
    with np.errstate(over="ignore"):
        s = (np.abs(g).max(-1, keepdims=True) * np.float32(1.0 / 127.0)).astype(np.float16)
    s = s.clip(-65504, 65504).astype(np.float64)
    code = np.rint(g.astype(np.float64) / np.where(s > 0, s, 1)).clip(-127, 127)
    return (code * s).reshape(np.shape(x))


def zero_points(k):
    """|zero point| of every dim's group of 32."""
    g = np.asarray(k, np.float64).reshape(*k.shape[:-1], -1, 32)
    return np.abs(np.repeat(g.min(-1, keepdims=True), 32, -1)).reshape(k.shape)


def sees(p, n, window, sinks):
    """Which of n tokens the token at place p sees."""
    t = np.arange(n)
    see = t <= p
    return see & ((t > p - window) | (t < sinks)) if window else see


def rows(q, k, v, places, window, sinks, scale, spread=None):
    """Attention in 64 bits of q [m][nq][d] at the places over k, v [n][H][d]: out, lse,
    sum p |v|, and the largest sum |q k| of a row's visible tokens (with `spread` added to
    |k|)."""
    m, nq, d = q.shape
    H = k.shape[1]
    out, lse, mass, reach = np.zeros((m, nq, d)), np.full((m, nq), -np.inf), np.zeros((m, nq, d)), np.zeros((m, nq))
    wide = np.abs(k) if spread is None else np.abs(k) + spread
    for i in range(m):
        see = sees(places[i], k.shape[0], window, sinks)
        if not see.any():
            continue
        for j in range(nq):
            h = j // (nq // H)
            s = scale * (k[see, h] @ q[i, j])
            reach[i, j] = abs(scale) * (wide[see, h] @ np.abs(q[i, j])).max()
            e = np.exp(s - s.max())
            w = e / e.sum()
            out[i, j], mass[i, j] = w @ v[see, h], w @ np.abs(v[see, h])
            lse[i, j] = s.max() + np.log(e.sum())
    return out, lse, mass, reach


def join(out, lse, mass, base_out, base_lse):
    top = np.maximum(lse, base_lse)
    ref = np.where(np.isfinite(top), top, 0.0)
    wa, wb = np.exp(lse - ref), np.exp(base_lse - ref)
    tot = np.where(wa + wb > 0, wa + wb, 1.0)
    out = (wa[..., None] * out + wb[..., None] * base_out) / tot[..., None]
    mass = (wa[..., None] * mass + wb[..., None] * np.abs(base_out)) / tot[..., None]
    return out, np.where(np.isfinite(top), ref + np.log(tot), -np.inf), mass


def check(out, lse, ref, ref_lse, mass, reach, weights):
    """out: a bf16 rounding of the result (2^-8 of the value), weights off by `weights`
    of themselves, and by what their scores are off: fp32 sums of up to 128 products in
    any order, at most 131 roundings (cut off: 2^-23 each) of partial sums of at most
    `reach`, 2^-15.9 of it; scaling, maximum, exponent and the hardware's exponential add
    5 roundings of the score and 2^-21.  lse: the same, and an fp32 logarithm of a sum
    of positive terms (2^-20)."""
    off = 2.0 ** -15.9 * reach + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(ref) + (weights + 2 * off[..., None]) * mass + 1e-30
    err = np.abs(out - ref)
    assert np.all(err <= tol), "out: worst %.3g of its tolerance" % (err / tol).max()
    none = ~np.isfinite(ref_lse)
    assert np.array_equal(lse[none], ref_lse[none])
    tol = off[~none] + 2.0 ** -20 * (1 + np.abs(ref_lse[~none]))
    err = np.abs(lse[~none] - ref_lse[~none])
    assert np.all(err <= tol), "lse: worst %.3g of its tolerance" % (err / tol).max()


class Pages:
    """A container full of NaN patterns and its table of scattered pages.  The table
    has -7 where no token is, and where `unseen` says that no query sees one."""

    def __init__(self, fmt, H, d, page, lens, seed=0, L=1, layer=0, max_pages=None, spare=2):
        self.fmt, self.H, self.d, self.P, self.lens, self.layer = fmt, H, d, page, list(lens), layer
        need = [(n + page - 1) // page for n in lens]
        self.max_pages = max_pages or max(1, max(need))
        self.n_pages = sum(need) + spare
        self.cfg = (L, H, d, page, self.n_pages, FORMATS[fmt])
        self.buf = Guarded(kv.kvpages_bytes(self.cfg), fill=0xFF)
        assert kv.kvpages_init(self.cfg, self.buf.t, self.buf.nbytes) == kv.KVP_OK
        ids = np.random.default_rng(seed).permutation(self.n_pages)
        self.table = np.full((len(lens), self.max_pages), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at: at + n]
            at += n
        self.slots = torch.tensor([int(self.table[b, t // page]) * page + t % page for b, n in enumerate(lens)
                                   for t in range(n)], dtype=torch.int64, device="cuda")
        self.lens_d = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.table_d = torch.from_numpy(self.table).cuda()

    def forget(self, m, window, sinks):
        """Takes the pages that hold no token which one of m queries sees from the table."""
        for b, n in enumerate(self.lens):
            any_sees = np.zeros(max(n, 1), bool)
            for i in range(m):
                any_sees[:n] |= sees(n - m + i, n, window, sinks)
            for p in range((n + self.P - 1) // self.P):
                if not any_sees[p * self.P:min(n, (p + 1) * self.P)].any():
                    self.table[b, p] = -7
        self.table_d = torch.from_numpy(self.table).cuda()

    def write(self, k, v):
        n = k.shape[0]
        ko, vo = (Guarded(max(16, n * self.H * self.d * 2)) for _ in range(2))
        rc = kv.kvpages_append(self.buf.t, self.cfg, self.layer, n, 0, None, k, v, self.slots, None, None, None, 0.0, 0, None,
                               None, ko.t, vo.t)
        assert rc == kv.KVP_OK, kv.kvp_strerror(rc)
        torch.cuda.synchronize()
        assert self.buf.canary_ok() and ko.canary_ok() and vo.canary_ok()
        return f64(ko.bf16((n, self.H, self.d))), f64(vo.bf16((n, self.H, self.d)))

    def read(self, max_tokens=None):
        T = max(1, max(self.lens)) if max_tokens is None else max_tokens
        shape = (len(self.lens), self.H, T, self.d)
        ko, vo = (Guarded(int(np.prod(shape)) * 2, fill=0x7F) for _ in range(2))
        rc = kv.kvpages_read(self.buf.t, self.cfg, self.layer, len(self.lens), self.table_d, self.max_pages, self.lens_d,
                             T, ko.t, vo.t)
        assert rc == kv.KVP_OK, kv.kvp_strerror(rc)
        torch.cuda.synchronize()
        assert ko.canary_ok() and vo.canary_ok()
        return f64(ko.bf16(shape)), f64(vo.bf16(shape))

    def attend(self, q, scale, window=0, sinks=0, base_out=None, base_lse=None, stream=None, plain=False):
        B, m, nq, d = q.shape
        out, lse = Guarded(q.numel() * 2, fill=0x7F), Guarded(B * m * nq * 4, fill=0x7F)
        wsb = kv.kvpages_attend_workspace_bytes(self.cfg, B, m, nq)
        ws = Guarded(wsb, fill=0xFF)
        first = (self.buf.t, self.cfg, self.layer, B, m, nq, q, scale)
        last = (self.table_d, self.max_pages, self.lens_d, base_out, base_lse, out.t, lse.t, ws.t, wsb, stream)
        rc = kv.kvpages_attend(*first, *last) if plain else kv.kvpages_attend_window(*first, window, sinks, *last)
        assert rc == kv.KVP_OK, kv.kvp_strerror(rc)
        torch.cuda.synchronize()
        assert out.canary_ok() and lse.canary_ok() and ws.canary_ok() and self.buf.canary_ok()
        return f64(out.bf16(q.shape)), lse.t.view(torch.float32).view(B, m, nq).cpu().numpy().astype(np.float64)

    def status(self):
        return kv.kvpages_status(self.buf.t)


def split(x, lens):
    cut = np.cumsum([0] + list(lens))
    return [x[cut[i]: cut[i + 1]] for i in range(len(lens))]


def prompt(q, k, v, n_first, window, sinks, scale):
    """As rows(), of a whole sequence's new tokens q [n][nq][d] at places n_first ...: by
    matrix products."""
    n, nq, d = q.shape
    T, H = k.shape[:2]
    out, lse, mass, reach = np.zeros((n, nq, d)), np.full((n, nq), -np.inf), np.zeros((n, nq, d)), np.zeros((n, nq))
    if not T or not n:
        return out, lse, mass, reach
    p, t = n_first + np.arange(n)[:, None], np.arange(T)[None, :]
    see = t <= p
    if window:
        see &= (t > p - window) | (t < sinks)
    some = see.any(1)
    for j in range(nq):
        h = j // (nq // H)
        kh, vh = np.where(np.isfinite(k[:, h]), k[:, h], 0), np.where(np.isfinite(v[:, h]), v[:, h], 0)
        s = np.where(see, scale * (q[:, j] @ kh.T), -np.inf)
        reach[:, j] = np.where(see, abs(scale) * (np.abs(q[:, j]) @ np.abs(kh).T), 0).max(1)
        top = np.where(some, s.max(1), 0)
        e = np.exp(s - top[:, None])
        tot = np.where(some, e.sum(1), 1)
        w = e / tot[:, None]
        out[:, j], mass[:, j] = w @ vh, w @ np.abs(vh)
        lse[:, j] = np.where(some, top + np.log(tot), -np.inf)
    return out, lse, mass, reach
