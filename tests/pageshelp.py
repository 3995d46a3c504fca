"""Plain 64-bit page cache: the definitions of include/kvpool.h's page
operators over dictionaries and numpy arrays, for comparison with the CUDA
path.  Shares no code with the library."""
import numpy as np

FORMATS = {"bf16": 0, "k8v8": 1, "k8v4": 2}


def f64(bits16):
    """bf16 bit patterns as float64."""
    return (np.asarray(bits16, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def to_bf16(x):
    """float64 -> nearest-even bf16, as float64 (through fp32: exact for the values compared here)."""
    b = np.asarray(x, np.float64).astype(np.float32).view(np.uint32)
    r = (b + 0x7FFF + ((b >> 16) & 1)) & np.uint32(0xFFFF0000)
    return r.view(np.float32).astype(np.float64)


def held8(x):
    """(values, scales) an 8-bit group format holds for fp32 x [..., d]."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], -1, 32)
    s = (np.abs(g).max(-1, keepdims=True) * np.float32(1.0 / 127.0)).astype(np.float16).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.where(s > 0, np.rint(g / s), np.float32(0)).clip(-127, 127)
    return (code.astype(np.float64) * s).reshape(x.shape), s[..., 0]


def held4(x):
    """Values the 4-bit format holds for fp32 x [..., d]."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], -1, 32)
    lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
    with np.errstate(over="ignore"):  # beyond fp16: held at its largest value
        s = ((hi - lo) * np.float32(1.0 / 15.0)).astype(np.float16).clip(-65504, 65504).astype(np.float64)
        z = lo.astype(np.float16).clip(-65504, 65504).astype(np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.where(s > 0, np.rint((g.astype(np.float64) - z) / s), 0.0).clip(0, 15)
    # the value is code * s + z rounded once to fp32
    return (code * s + z).astype(np.float32).astype(np.float64).reshape(x.shape)


def held(x, fmt, values):
    if fmt == "bf16":
        return to_bf16(x)
    return held4(x) if values and fmt == "k8v4" else held8(x)[0]


def heads(x, weight, eps, positions, inv_freq, rot):
    """Norm and rotation of [n, heads, d] in 64 bits."""
    y = np.array(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    if rot:
        h = rot // 2
        ang = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float32).astype(np.float64)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        a, b = y[..., :h].copy(), y[..., h:rot].copy()
        y[..., :h], y[..., h:rot] = a * c - b * s, b * c + a * s
    return y


def attend(q, k, v, lens, scale, base_out=None, base_lse=None):
    """q [B][m][nq][d]; k, v: lists of [len][H][d]; float64 out, lse, and
    sum p |v| and sum p max|q.k| terms for tolerances."""
    B, m, nq, d = q.shape
    out, lse = np.zeros((B, m, nq, d)), np.full((B, m, nq), -np.inf)
    mass = np.zeros((B, m, nq, d))
    reach = np.zeros((B, m, nq))
    for b in range(B):
        H = k[b].shape[1]
        for i in range(m):
            n = max(0, lens[b] - (m - 1 - i))
            if n:
                for j in range(nq):
                    h = j // (nq // H)
                    s = scale * (k[b][:n, h] @ q[b, i, j])
                    reach[b, i, j] = abs(scale) * (np.abs(k[b][:n, h]) @ np.abs(q[b, i, j])).max()
                    e = np.exp(s - s.max())
                    out[b, i, j] = (e / e.sum()) @ v[b][:n, h]
                    mass[b, i, j] = (e / e.sum()) @ np.abs(v[b][:n, h])
                    lse[b, i, j] = s.max() + np.log(e.sum())
    if base_out is not None:
        top = np.maximum(lse, base_lse)
        ref = np.where(np.isfinite(top), top, 0.0)
        wa, wb = np.exp(lse - ref), np.exp(base_lse - ref)
        tot = np.where(wa + wb > 0, wa + wb, 1.0)
        out = (wa[..., None] * out + wb[..., None] * base_out) / tot[..., None]
        mass = (wa[..., None] * mass + wb[..., None] * np.abs(base_out)) / tot[..., None]
        lse = np.where(np.isfinite(top), ref + np.log(tot), -np.inf)
    return out, lse, mass, reach
