"""Host-side checks of the 4-bit page format, of positions with several axes and of
windows that need no GPU: sizes, and every refusal before any work is enqueued."""
import ctypes

import pytest
import torch

import agent_shared_compressed_gb300 as kv
from agent_shared_compressed_gb300 import build as kvbuild

OK = 0x10000
CFG = (2, 4, 128, 32, 8, kv.KVP_PAGES_K4V4)


@pytest.fixture(scope="module", autouse=True)
def built():
    kvbuild.build()
    kv.load()


@pytest.mark.parametrize("d", [64, 128])
def test_container_bytes(d):
    """Per token and head: 4 bits a dim, and a scale and a zero point of 2 bytes for every
    32 of them, of keys and of values."""
    for L, H, page, n in [(1, 1, 16, 1), (3, 5, 32, 7), (32, 8, 1024, 40)]:
        layer = n * page * H * (d + 8 * (d // 32))
        assert kv.kvpages_bytes((L, H, d, page, n, kv.KVP_PAGES_K4V4)) == 256 + L * ((layer + 255) // 256 * 256)
    assert kv.kvpages_bytes((1, 1, d, 16, 1, 3)) == kv.kvpages_bytes((1, 1, d, 16, 1, 5)) == 0


def test_append_axes_refusals():
    w, r, ax = [1.0] * 64, kv.rows(OK, 512, 128), [i % 3 for i in range(64)]

    def call(n=3, pos=OK, n_axes=3, axes=ax, rot=128, freq=w, cfg=CFG, nq=8, slots=OK, pages=OK, qo=OK):
        return kv.kvpages_append_axes(pages, cfg, 0, n, nq, r, r, r, slots, pos, n_axes, axes, None, None, 0.0, rot, freq, qo,
                                      None, None)

    assert call(n_axes=0) == call(n_axes=kv.KVP_MAX_AXES + 1) == call(n_axes=2) == kv.KVP_ERR_ARG   # axis 2 of two
    assert call(axes=None) == call(pos=None) == call(freq=None) == call(axes=[0] * 63 + [3]) == kv.KVP_ERR_ARG
    assert call(rot=32) == call(pages=None) == call(slots=None) == call(qo=None) == kv.KVP_ERR_ARG
    assert call(pos=OK + 4) == call(qo=OK + 8) == kv.KVP_ERR_ALIGN
    assert call(n=0) == kv.KVP_OK
    assert call(n=0, rot=0, axes=None, pos=None, freq=None) == kv.KVP_OK
    assert call(n=0, rot=64, axes=[4] * 32 + [0]) == kv.KVP_ERR_ARG and call(n=0, rot=64, axes=[2] * 32) == kv.KVP_OK
    with pytest.raises(ValueError):
        call(axes=[0] * 63)
    with pytest.raises(ValueError):
        call(axes=[-1] * 64)
    with pytest.raises(ValueError):
        call(axes=(ctypes.c_int * 64)())
    with pytest.raises(ValueError):  # two axes' positions for three
        call(pos=torch.zeros(2, 3, dtype=torch.int64))
    with pytest.raises(ValueError):
        call(pos=torch.zeros(3, 6, dtype=torch.int64)[:, ::2])


def test_attend_window_refusals():
    ws = kv.kvpages_attend_workspace_bytes(CFG, 2, 3, 8)

    def call(pages=OK, layer=0, n=2, m=3, nq=8, q=OK, scale=1.0, window=16, sinks=4, table=OK, mp=4, lens=OK, bo=None, bl=None,
             out=OK, lse=OK, w=OK, wb=ws):
        return kv.kvpages_attend_window(pages, CFG, layer, n, m, nq, q, scale, window, sinks, table, mp, lens, bo, bl, out, lse, w, wb)

    assert call(window=-1) == call(sinks=-1) == call(window=0, sinks=-2) == kv.KVP_ERR_ARG
    assert call(pages=None) == call(layer=2) == call(m=0) == call(nq=6) == call(q=None) == call(bo=OK) == kv.KVP_ERR_ARG
    assert call(scale=float("nan")) == kv.KVP_ERR_ARG and call(m=65) == call(wb=ws - 1) == kv.KVP_ERR_SIZE
    assert call(q=OK + 8) == call(out=OK + 8) == kv.KVP_ERR_ALIGN
    big = 2 ** 31 - 1
    assert call(n=0) == call(n=0, window=big, sinks=big) == call(n=0, window=0, sinks=0) == kv.KVP_OK
    cfg = kv.PagesConfig(*CFG)
    for bad in (dict(q=torch.zeros(2, 3, 8, 128)), dict(table=torch.zeros(2, 3, dtype=torch.int32)),
                dict(lens=torch.zeros(2, dtype=torch.int64)), dict(out=torch.zeros(2, 3, 8, 64, dtype=torch.bfloat16)),
                dict(w=torch.zeros(ws - 1, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call(**bad)
    assert cfg.format == kv.KVP_PAGES_K4V4


def test_no_read_only_loads_of_what_may_be_written():
    """The kernels that may be resident while the one before them runs read what it writes: no
    loads of the kind that wants memory nobody writes meanwhile (as the other page kernels)."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "agent_shared_compressed_gb300", "csrc")
    for name in ("kvpages_attend.cuh", "kvprompt.cu"):
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(os.path.join(csrc, name)).read(), flags=re.S)
        assert not re.findall(r"\b__ldg\b|\b__ldc[agsv]\b|\.nc\b|\bld_stream_\w+|\bld_v4_policy\b|__restrict__", code), name
        assert "griddepcontrol.wait;" in code
