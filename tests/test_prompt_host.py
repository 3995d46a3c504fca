"""Host-side checks of attention of whole prompts that need no GPU: every refusal
before any work is enqueued, and tensors that do not hold what a call reads."""
import pytest
import torch

import agent_shared_compressed_gb300 as kv
from agent_shared_compressed_gb300 import build as kvbuild

OK = 0x10000
SHAPE = (2, 5, 9, 8, 4, 128)
R, RK = kv.rows(OK, 1024, 128), kv.rows(OK, 512, 128)


@pytest.fixture(scope="module", autouse=True)
def built():
    kvbuild.build()
    kv.load()


def call(shape=SHAPE, q=R, k=RK, v=RK, qf=OK, kf=OK, kl=OK, scale=1.0, window=0, sinks=0, bo=None, bl=None, out=OK, lse=OK,
         err=OK, ws=OK, wb=None):
    return kv.kvprompt_attend(shape, q, k, v, qf, kf, kl, scale, window, sinks, bo, bl, out, lse, err, ws,
                              max(kv.kvprompt_workspace_bytes(shape), 1) if wb is None else wb)


@pytest.mark.parametrize("shape,code", [
    ((-1, 5, 9, 8, 4, 128), kv.KVP_ERR_ARG), ((2, -5, 9, 8, 4, 128), kv.KVP_ERR_ARG), ((2, 5, -9, 8, 4, 128), kv.KVP_ERR_ARG),
    ((2, 5, 9, 0, 4, 128), kv.KVP_ERR_ARG), ((2, 5, 9, 8, 0, 128), kv.KVP_ERR_ARG), ((2, 5, 9, 9, 4, 128), kv.KVP_ERR_ARG),
    ((2, 5, 9, 8, 4, 96), kv.KVP_ERR_UNSUPPORTED_D), ((2, 5, 9, 8, 4, 256), kv.KVP_ERR_UNSUPPORTED_D),
    ((kv.KVP_PROMPT_MAX_SEQS + 1, 5, 9, 8, 4, 128), kv.KVP_ERR_SIZE), ((2, 5, 9, 129, 1, 128), kv.KVP_ERR_SIZE),
    ((2, 1 << 28, 9, 8, 4, 128), kv.KVP_ERR_SIZE), ((2, 5, 9, 1 << 17, 1 << 17, 64), kv.KVP_ERR_SIZE)])
def test_invalid_shapes(shape, code):
    assert kv.kvprompt_workspace_bytes(shape) == 0
    assert call(shape=shape) == code


def test_refusals():
    assert call(window=-1) == call(sinks=-1) == call(scale=float("nan")) == call(scale=float("inf")) == kv.KVP_ERR_ARG
    assert call(q=None) == call(k=None) == call(v=None) == call(qf=None) == call(kf=None) == call(kl=None) == kv.KVP_ERR_ARG
    assert call(out=None) == call(ws=None) == call(bo=OK) == call(bl=OK) == call(k=kv.Rows(None, 512, 128)) == kv.KVP_ERR_ARG
    assert call(wb=kv.kvprompt_workspace_bytes(SHAPE) - 1) == kv.KVP_ERR_SIZE
    for bad in (dict(q=kv.rows(OK + 8, 1024, 128)), dict(k=kv.rows(OK, 516, 128)), dict(v=kv.rows(OK, 512, 132)), dict(qf=OK + 2),
                dict(kf=OK + 2), dict(kl=OK + 1), dict(bo=OK + 8, bl=OK), dict(bo=OK, bl=OK + 2), dict(out=OK + 8),
                dict(lse=OK + 2), dict(err=OK + 2), dict(ws=OK + 8)):
        assert call(**bad) == kv.KVP_ERR_ALIGN, bad
    # strides of several tokens or heads are positive and below 2^38; of one they say nothing
    for bad in (dict(q=kv.rows(OK, 0, 128)), dict(q=kv.rows(OK, -1024, 128)), dict(k=kv.rows(OK, 512, 0)),
                dict(v=kv.rows(OK, 512, -128)), dict(k=kv.rows(OK, 1 << 38, 128)), dict(v=kv.rows(OK, 512, 1 << 38))):
        assert call(**bad) == kv.KVP_ERR_ARG, bad
    assert call(shape=(0, 1, 1, 1, 1, 128), q=kv.rows(OK, 0, -8), k=kv.rows(OK, -8, 0), v=kv.rows(OK, 0, 0)) == kv.KVP_OK
    # nothing to do, nothing launched
    n = kv.kvp_launch_count()
    assert call(shape=(0, 5, 9, 8, 4, 128)) == call(shape=(2, 0, 9, 8, 4, 128), q=kv.Rows(None, 1024, 128)) == kv.KVP_OK
    assert kv.kvp_launch_count() == n
    assert kv.kvprompt_status(None) == kv.KVP_ERR_ARG and kv.kvprompt_status(OK + 2) == kv.KVP_ERR_ALIGN


def test_tensors_that_do_not_hold_it():
    x = torch.zeros(9, 16, 128, dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    for bad in (dict(q=x[:4, :8]), dict(q=x[:5, :7]), dict(q=x[:5, :8].float()), dict(k=x[:8, :4]), dict(v=x[:, :4, :64]),
                dict(k=x.transpose(1, 2)[:, :4]), dict(qf=torch.zeros(2, **i32)), dict(kf=torch.zeros(1, **i32)),
                dict(kl=torch.zeros(2, dtype=torch.int64)), dict(out=torch.zeros(5, 8, 127, dtype=torch.bfloat16)),
                dict(lse=torch.zeros(5, 7)), dict(bo=torch.zeros(5, 8, 128), bl=torch.zeros(39)),
                dict(err=torch.zeros(1, dtype=torch.int64)), dict(ws=torch.zeros(16, dtype=torch.uint8), wb=17)):
        with pytest.raises(ValueError):
            call(**bad)


def test_tensors_without_elements():
    """No new tokens, or no keys: such a tensor's strides say nothing (one made from an empty
    numpy array has strides of 0)."""
    for empty in (torch.empty(0, 8, 128, dtype=torch.bfloat16),
                  torch.as_strided(torch.empty(1, dtype=torch.bfloat16), (0, 8, 128), (0, 0, 0))):
        assert call(shape=(2, 0, 9, 8, 4, 128), q=empty) == kv.KVP_OK
        assert call(shape=(2, 0, 0, 8, 4, 128), q=empty, k=empty[:, :4], v=empty[:, :4]) == kv.KVP_OK
        r = kv.rows(empty)
        assert (r.token_stride, r.head_stride) == (1024, 128)
        with pytest.raises(ValueError):
            call(shape=(2, 1, 9, 8, 4, 128), q=empty)
