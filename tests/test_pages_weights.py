"""The probe of the weights' precision (pagesweights.py) tells a sum of two bf16
from one bf16 and from 11 bits: mistakes planted in the plain form (no GPU needed)."""
import numpy as np
import pytest

import pageshelp as P
import pagesweights as W

ROUNDINGS = {"two bf16": lambda e: P.to_bf16(e) + P.to_bf16(e - P.to_bf16(e)), "bf16": P.to_bf16,
             "fp16": lambda e: e.astype(np.float16).astype(np.float64),
             "fp32": lambda e: e.astype(np.float32).astype(np.float64)}


@pytest.mark.parametrize("fmt", ["bf16", "k8v8", "k8v4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("repeat", [1, 20, 400])
def test_probe_tells_roundings_apart(fmt, d, repeat):
    q, k, v, scale = W.sequence(fmt, d, repeat, 16)
    hk, hv = P.held(k, fmt, False), P.held(v, fmt, True)
    ref, _, mass, reach = P.attend(q[None, None], [hk], [hv], [len(k)], scale)
    tol = W.bound(ref, mass, reach[..., None], repeat)[0, 0]
    for name, rounding in ROUNDINGS.items():
        worst = (np.abs(W.with_rounded_weights(q, hk, hv, scale, rounding) - ref[0, 0]) / tol).max()
        assert worst <= 0.5 if name in ("two bf16", "fp32") else worst > 2, (name, worst)
