"""Host-side checks of the page container's entry points that need no GPU:
sizes against the format, and every refusal, each before any work is enqueued."""
import numpy as np
import pytest

import agent_shared_compressed_gb300 as kv
from agent_shared_compressed_gb300 import build as kvbuild
import pageshelp as P

OK = 0x10000
CFG = (2, 4, 128, 32, 8, kv.KVP_PAGES_K8V8)


@pytest.fixture(scope="module", autouse=True)
def built():
    kvbuild.build()
    kv.load()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt,bits", [("bf16", 32), ("k8v8", 16 + 1), ("k8v4", 12 + 0.5 + 1)])
def test_container_bytes(d, fmt, bits):
    """Per (token, head): codes of d keys and d values, 2-byte scales of every
    32 (4-bit values: scale and zero point); bits per dim given above."""
    for L, H, page, n in [(1, 1, 16, 1), (3, 5, 32, 7), (32, 8, 1024, 40)]:
        layer = n * page * H * int(d * bits) // 8
        want = 256 + L * ((layer + 255) // 256 * 256)
        assert kv.kvpages_bytes((L, H, d, page, n, P.FORMATS[fmt])) == want


@pytest.mark.parametrize("cfg,code", [
    ((0, 4, 128, 32, 8, 1), kv.KVP_ERR_ARG), ((2, 0, 128, 32, 8, 1), kv.KVP_ERR_ARG),
    ((2, 4, 96, 32, 8, 1), kv.KVP_ERR_UNSUPPORTED_D), ((2, 4, 128, 24, 8, 1), kv.KVP_ERR_ARG),
    ((2, 4, 128, 8, 8, 1), kv.KVP_ERR_ARG), ((2, 4, 128, 2048, 8, 1), kv.KVP_ERR_ARG),
    ((2, 4, 128, 32, 0, 1), kv.KVP_ERR_ARG), ((2, 4, 128, 32, 8, 3), kv.KVP_ERR_ARG),
    ((2, 4, 128, 32, 8, -1), kv.KVP_ERR_ARG), ((513, 4, 128, 32, 8, 1), kv.KVP_ERR_SIZE),
    ((2, 4097, 128, 32, 8, 1), kv.KVP_ERR_SIZE), ((512, 4096, 128, 1024, 2 ** 31 - 1, 0), kv.KVP_ERR_SIZE)])
def test_invalid_configurations(cfg, code):
    assert kv.kvpages_bytes(cfg) == 0
    assert kv.kvpages_attend_workspace_bytes(cfg, 1, 1, 4) == 0
    assert kv.kvpages_init(cfg, OK, 1 << 40) == code
    r = kv.rows(OK, 512, 128)
    assert kv.kvpages_append(OK, cfg, 0, 1, 0, None, r, r, OK, None, None, None, 0.0, 0, None, None, None, None) == code
    assert kv.kvpages_read(OK, cfg, 0, 1, OK, 1, OK, 1, OK, OK) == code
    assert kv.kvpages_attend(OK, cfg, 0, 1, 1, 4, OK, 1.0, OK, 1, OK, None, None, OK, OK, OK, 1 << 30) == code


def test_init_and_status_refusals():
    n = kv.kvpages_bytes(CFG)
    assert kv.kvpages_init(CFG, None, n) == kv.KVP_ERR_ARG
    assert kv.kvpages_init(CFG, OK + 128, n) == kv.KVP_ERR_ALIGN
    assert kv.kvpages_init(CFG, OK, n - 1) == kv.KVP_ERR_SIZE
    assert kv.kvpages_status(None) == kv.KVP_ERR_ARG
    assert kv.kvp_strerror(kv.KVP_ERR_PAGE) != "unknown status"


def test_append_refusals():
    w = [1.0] * 64
    r = kv.rows(OK, 512, 128)

    def call(pages=OK, layer=0, n=3, nq=8, q=r, k=r, v=r, slots=OK, pos=OK, qn=None, kn=None, eps=1e-5, rot=128, freq=w,
             qo=OK, ko=None, vo=None):
        return kv.kvpages_append(pages, CFG, layer, n, nq, q, k, v, slots, pos, qn, kn, eps, rot, freq, qo, ko, vo)

    assert call(pages=None) == call(layer=2) == call(layer=-1) == call(n=-1) == call(nq=-1) == kv.KVP_ERR_ARG
    assert call(q=None) == call(k=None) == call(v=None) == call(slots=None) == call(qo=None) == kv.KVP_ERR_ARG
    assert call(k=kv.Rows(None, 512, 128)) == kv.KVP_ERR_ARG
    assert call(pos=None) == call(freq=None) == kv.KVP_ERR_ARG
    assert call(rot=32) == call(rot=96) == call(rot=-64) == kv.KVP_ERR_ARG
    assert call(freq=w[:-1] + [float("inf")]) == call(freq=w[:-1] + [float("nan")]) == kv.KVP_ERR_ARG
    assert call(qn=OK, eps=float("nan")) == call(kn=OK, eps=-1.0) == kv.KVP_ERR_ARG
    assert call(nq=65537) == kv.KVP_ERR_SIZE
    for bad in (dict(pages=OK + 16), dict(q=kv.rows(OK + 8, 512, 128)), dict(k=kv.rows(OK, 516, 128)),
                dict(v=kv.rows(OK, 512, 132)), dict(slots=OK + 4), dict(pos=OK + 4), dict(qn=OK + 8), dict(kn=OK + 8),
                dict(qo=OK + 8), dict(ko=OK + 8), dict(vo=OK + 8)):
        assert call(**bad) == kv.KVP_ERR_ALIGN, bad
    # head_dim 64 takes no 128-dim rotation
    c64 = (2, 4, 64, 32, 8, 1)
    assert kv.kvpages_append(OK, c64, 0, 3, 8, r, r, r, OK, OK, None, None, 0.0, 128, w, OK, None, None) == kv.KVP_ERR_ARG
    assert call(n=0) == kv.KVP_OK                                      # nothing to do, nothing launched


def test_rows_of_tensors():
    import torch
    x = torch.zeros(5, 7, 128, dtype=torch.bfloat16)
    r = kv.rows(x[:, 2:4])
    assert (r.ptr, r.token_stride, r.head_stride) == (x.data_ptr() + 2 * 128 * 2, 7 * 128, 128)
    r = kv.rows(x.transpose(0, 1))
    assert (r.token_stride, r.head_stride) == (128, 7 * 128)
    with pytest.raises(ValueError):
        kv.rows(x.transpose(1, 2))


def test_read_refusals():
    def call(pages=OK, layer=0, n=2, table=OK, mp=4, lens=OK, mt=64, k=OK, v=OK):
        return kv.kvpages_read(pages, CFG, layer, n, table, mp, lens, mt, k, v)

    assert call(pages=None) == call(layer=2) == call(n=-1) == call(mp=0) == call(mt=0) == kv.KVP_ERR_ARG
    assert call(table=None) == call(lens=None) == call(k=None) == call(v=None) == kv.KVP_ERR_ARG
    assert call(pages=OK + 64) == call(table=OK + 2) == call(lens=OK + 1) == call(k=OK + 8) == kv.KVP_ERR_ALIGN
    assert call(n=2 ** 30) == kv.KVP_ERR_SIZE
    assert call(n=0) == kv.KVP_OK


def test_attend_refusals():
    ws = kv.kvpages_attend_workspace_bytes(CFG, 2, 3, 8)
    assert ws > 0
    assert kv.kvpages_attend_workspace_bytes(CFG, 2, 3, 6) == 0

    def call(pages=OK, layer=0, n=2, m=3, nq=8, q=OK, scale=1.0, table=OK, mp=4, lens=OK, bo=None, bl=None, out=OK, lse=OK,
             w=OK, wb=None):
        return kv.kvpages_attend(pages, CFG, layer, n, m, nq, q, scale, table, mp, lens, bo, bl, out, lse, w,
                                 ws if wb is None else wb)

    assert call(pages=None) == call(layer=2) == call(n=-1) == call(m=0) == call(nq=6) == call(nq=0) == kv.KVP_ERR_ARG
    assert call(mp=0) == call(q=None) == call(table=None) == call(lens=None) == call(out=None) == kv.KVP_ERR_ARG
    assert call(w=None) == call(bo=OK) == call(bl=OK) == kv.KVP_ERR_ARG
    assert call(scale=float("nan")) == call(scale=float("inf")) == kv.KVP_ERR_ARG
    assert call(m=65) == call(n=kv.KVP_PAGES_MAX_SEQS + 1) == call(wb=ws - 1) == kv.KVP_ERR_SIZE
    assert call(mp=2 ** 31 - 1) == kv.KVP_ERR_SIZE                     # 2^35 tokens or more
    for bad in (dict(pages=OK + 128), dict(q=OK + 8), dict(table=OK + 2), dict(lens=OK + 2), dict(out=OK + 8),
                dict(lse=OK + 2), dict(w=OK + 8), dict(bo=OK + 8, bl=OK), dict(bo=OK, bl=OK + 2)):
        assert call(**bad) == kv.KVP_ERR_ALIGN, bad
    assert call(n=0) == kv.KVP_OK


def test_plain_formats():
    """The plain forms themselves: the groups' extremes are held to half a step."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 4, 64)).astype(np.float32)
    h, s = P.held8(x)
    assert np.all(np.abs(h - x).reshape(50, 4, 2, 32) <= 0.5 * s[..., None] * 1.0001)
    g = x.reshape(50, 4, 2, 32)
    step = (g.max(-1) - g.min(-1)) / 15
    assert np.all(np.abs(P.held4(x) - x).reshape(50, 4, 2, 32) <= step[..., None] * (0.5 + 2.0 ** -6))
    assert np.array_equal(P.held8(np.zeros((1, 1, 64)))[0], np.zeros((1, 1, 64)))
    assert np.array_equal(P.held4(np.full((1, 1, 64), 1.5)), np.full((1, 1, 64), 1.5))
