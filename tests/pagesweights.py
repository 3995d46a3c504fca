"""A sequence whose attention is the difference of two equal terms, so that what is
left over shows how exactly the weights were held; and the bound that goes with it."""
import numpy as np

import pageshelp as P

# two values of a dim are c s and -c S for the same codes c: of bf16, with 4 bits each
# for c and S; of 8-bit codes, with S the fp16 scale of a row whose largest is 175; of
# 4-bit codes about their middle
_TOPS = {"bf16": 1.375, "k8v8": 175.0, "k8v4": 1.375}


def sequence(fmt, d, repeat, n_rows, seed=0):
    """(q [rows][d], k, v [3 repeat][1][d], scale): tokens (a, b, c) repeated; a's and
    b's weighted values cancel in every dim, c has no value and takes another share of
    the softmax for every query row."""
    rng = np.random.default_rng(seed)
    k, v = np.zeros((3, d)), np.zeros((3, d))
    k[0, 0], k[1, 0], k[2, 1] = 1.0, 2.0, 1.0
    if fmt == "k8v4":
        c = rng.integers(0, 16, d) - 7.5
        c[::32], c[1::32] = -7.5, 7.5     # a group's extremes, hence its step
        v[0], v[1] = c, -c * _TOPS[fmt]
    elif fmt == "k8v8":
        c = rng.integers(-126, 127, d).astype(np.float64)
        c[::32] = 127.0
        v[0], v[1] = c, -P.to_bf16(c * np.float64(np.float16(np.float32(175.0) * np.float32(1.0 / 127.0))))
        v[1, ::32] = -175.0
    else:
        c = rng.integers(1, 16, d) * rng.choice([-1.0, 1.0], d)
        v[0], v[1] = c, -c * _TOPS[fmt]
    hk, hv = P.held(k[:, None], fmt, False)[:, 0], P.held(v[:, None], fmt, True)[:, 0]
    ratio = -hv[1, 0] / hv[0, 0]           # of a's weight to b's
    assert np.array_equal(hv[1], -hv[0] * ratio) or np.abs(hv[1] + hv[0] * ratio).max() <= 1e-12
    q = np.zeros((n_rows, d))
    q[:, 0] = -1.0
    q[:, 1] = P.to_bf16(3.0 * rng.standard_normal(n_rows))
    scale = float(np.float32(np.log(ratio) / (hk[1, 0] - hk[0, 0])))
    return q, np.tile(k, (repeat, 1))[:, None], np.tile(v, (repeat, 1))[:, None], scale


def bound(ref, mass, reach, steps):
    """bf16's half step of the result; 2^-17 of each weight; scores in fp32 (2^-19 of
    1 and of the largest sum of products); fp32 additions, `steps` one after the other."""
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -17 + 2.0 ** -19 * (1 + reach) + steps * 2.0 ** -23) * mass


def with_rounded_weights(q, k, v, scale, rounding):
    """Attention of rows q over [n][1][d], the weights rounded as given (the sum is not)."""
    out = np.zeros(q.shape)
    for j, x in enumerate(q):
        s = scale * (k[:, 0] @ x)
        e = np.exp(s - s.max())
        out[j] = rounding(e) @ v[:, 0] / e.sum()
    return out
