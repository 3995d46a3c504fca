"""The page calls of the binding refuse tensors that do not hold what the kernels
would read or write: another type, too few elements, another order.  A stand-in
for the library shows that nothing reaches it (no GPU needed)."""
import ctypes

import pytest
import torch

import agent_shared_compressed_gb300 as kv
from agent_shared_compressed_gb300 import binding

CFG = kv.PagesConfig(1, 2, 64, 16, 8, kv.KVP_PAGES_K8V8)
N, NQ, H, D, B, M, WIDTH, T = 3, 4, 2, 64, 2, 3, 5, 7


class Library:
    """Notes the calls that reach it."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or kv.KVP_OK


@pytest.fixture
def lib(monkeypatch):
    made = Library()
    monkeypatch.setattr(binding, "load", lambda path=None: made)
    return made


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def turned(x):
    """The same elements in another order of memory."""
    return x.transpose(0, 1).contiguous().transpose(0, 1)


def append(**change):
    a = dict(pages=torch.zeros(256, dtype=torch.uint8), cfg=CFG, layer=0, n_tokens=N, n_q_heads=NQ, q=bf16(N, NQ, D),
             k=bf16(N, H, D), v=bf16(N, H, D), slots=torch.zeros(N, dtype=torch.int64),
             positions=torch.zeros(N, dtype=torch.int64), q_norm=bf16(D), k_norm=bf16(D), eps=0.0, rot_dim=64,
             inv_freq=[1.0] * 32, q_out=bf16(N, NQ, D), k_out=bf16(N, H, D), v_out=bf16(N, H, D))
    return kv.kvpages_append(**dict(a, **change))


def read(**change):
    a = dict(pages=torch.zeros(256, dtype=torch.uint8), cfg=CFG, layer=0, n_seqs=B,
             table=torch.zeros(B, WIDTH, dtype=torch.int32), max_pages=WIDTH, lens=torch.zeros(B, dtype=torch.int32),
             max_tokens=T, k_dst=bf16(B, H, T, D), v_dst=bf16(B, H, T, D))
    return kv.kvpages_read(**dict(a, **change))


def attend(**change):
    a = dict(pages=torch.zeros(256, dtype=torch.uint8), cfg=CFG, layer=0, n_seqs=B, n_q_tokens=M, n_q_heads=NQ,
             q=bf16(B, M, NQ, D), scale=1.0, table=torch.zeros(B, WIDTH, dtype=torch.int32), max_pages=WIDTH,
             lens=torch.zeros(B, dtype=torch.int32), base_out=torch.zeros(B, M, NQ, D), base_lse=torch.zeros(B, M, NQ),
             out=bf16(B, M, NQ, D), lse=torch.zeros(B, M, NQ), ws=torch.zeros(4096, dtype=torch.uint8), ws_bytes=4096)
    return kv.kvpages_attend(**dict(a, **change))


def test_what_fits_is_passed_on(lib):
    assert append() == read() == attend() == kv.KVP_OK
    # more than needed, memory as bytes, addresses, what may be left out
    append(slots=torch.zeros(N + 1, dtype=torch.int64), q=bf16(N + 2, NQ, D), k_out=torch.zeros(N * H * D * 2, dtype=torch.uint8))
    append(k=bf16(H, N, D).transpose(0, 1), v=bf16(N, H + 6, D)[:, 2:2 + H], slots=64, positions=64, q_out=64)
    append(n_q_heads=0, q=None, q_out=None, positions=None, rot_dim=0, inv_freq=None, q_norm=None, k_norm=None, k_out=None, v_out=None)
    append(k=kv.rows(64, H * D, D), v=kv.rows(bf16(N, H, D)))
    attend(q=bf16(B, 1, M * NQ, D), base_out=None, base_lse=None, lse=None, out=torch.zeros(B * M * NQ * D * 2, dtype=torch.uint8))
    read(table=torch.zeros(B + 1, WIDTH, dtype=torch.int32), k_dst=64, v_dst=64)
    kv.kvpages_init(CFG, torch.zeros(512, dtype=torch.uint8), 512)
    assert len(lib.calls) == 10


def test_rows_reach_the_library_as_pointer_and_strides(lib):
    fused = bf16(N, NQ + 2 * H, D)
    k = fused[:, NQ:NQ + H]
    for form in (k, kv.rows(k)):
        lib.calls.clear()
        append(k=form)
        got = lib.calls[0][1][6]
        got = kv.Rows.from_buffer_copy(got) if isinstance(got, bytes) else kv.Rows.from_address(got)
        assert (got.ptr, got.token_stride, got.head_stride) == (k.data_ptr(), (NQ + 2 * H) * D, D)


@pytest.mark.parametrize("change", [
    dict(slots=torch.zeros(N, dtype=torch.int32)), dict(slots=torch.zeros(N - 1, dtype=torch.int64)),
    dict(slots=torch.zeros(2 * N, dtype=torch.int64)[::2]), dict(slots=torch.zeros(8 * N - 1, dtype=torch.uint8)),
    dict(positions=torch.zeros(N, dtype=torch.int32)), dict(positions=torch.zeros(N, dtype=torch.float64)),
    dict(q=torch.zeros(N, NQ, D)), dict(q=bf16(N - 1, NQ, D)), dict(q=bf16(N, NQ - 1, D)), dict(q=bf16(N, NQ, 2 * D)),
    dict(k=bf16(N, NQ, D)), dict(k=bf16(N, H, D).half()), dict(v=bf16(N, H + 1, D)), dict(v=bf16(N, H, D // 2)),
    dict(k=kv.rows(bf16(N - 1, H, D))), dict(v=kv.rows(bf16(N, H + 1, D))),
    dict(k=bf16(N, D, H).transpose(1, 2)),
    dict(q_norm=bf16(D - 1)), dict(k_norm=torch.zeros(D)), dict(q_out=bf16(N, NQ, D - 1)), dict(q_out=turned(bf16(N, NQ, D))),
    dict(k_out=torch.zeros(N, H, D)), dict(v_out=bf16(N, H - 1, D)), dict(v_out=turned(bf16(N, H, D)))])
def test_append_refuses(lib, change):
    with pytest.raises(ValueError):
        append(**change)
    assert not lib.calls


@pytest.mark.parametrize("change", [
    dict(table=torch.zeros(B, WIDTH, dtype=torch.int64)), dict(table=torch.zeros(WIDTH, B, dtype=torch.int32).t()),
    dict(table=torch.zeros(B, WIDTH - 1, dtype=torch.int32)), dict(table=torch.zeros(B, 2 * WIDTH, dtype=torch.int32)[:, :WIDTH]),
    dict(lens=torch.zeros(B, dtype=torch.int64)), dict(lens=torch.zeros(B - 1, dtype=torch.int32)),
    dict(k_dst=bf16(B, H, T - 1, D)), dict(v_dst=turned(bf16(B, H, T, D))), dict(v_dst=torch.zeros(B, H, T, D))])
def test_read_refuses(lib, change):
    with pytest.raises(ValueError):
        read(**change)
    assert not lib.calls


@pytest.mark.parametrize("change", [
    dict(q=torch.zeros(B, M, NQ, D)), dict(q=turned(bf16(B, M, NQ, D))), dict(q=bf16(B, M, NQ - 1, D)),
    dict(table=torch.zeros(B, WIDTH, dtype=torch.int64)), dict(table=torch.zeros(WIDTH, B, dtype=torch.int32).t()),
    dict(lens=torch.zeros(B, dtype=torch.int64)), dict(lens=torch.zeros(2 * B, dtype=torch.int32)[::2]),
    dict(base_out=bf16(B, M, NQ, D)), dict(base_lse=torch.zeros(B, M, NQ, dtype=torch.float64)),
    dict(base_lse=torch.zeros(B, M, NQ - 1)), dict(out=torch.zeros(B, M, NQ, D)), dict(out=turned(bf16(B, M, NQ, D))),
    dict(lse=torch.zeros(B, M, 1)), dict(lse=turned(torch.zeros(B, M, NQ))), dict(ws=torch.zeros(4095, dtype=torch.uint8)),
    dict(ws=torch.zeros(8192, dtype=torch.uint8)[::2])])
def test_attend_refuses(lib, change):
    with pytest.raises(ValueError):
        attend(**change)
    assert not lib.calls


def test_other_refusals(lib):
    with pytest.raises(ValueError):
        kv.kvpages_init(CFG, torch.zeros(511, dtype=torch.uint8), 512)
    with pytest.raises(ValueError):
        kv.rows(torch.zeros(N, H, D))
    with pytest.raises(TypeError):
        attend(lens="lens")
    assert not lib.calls


@pytest.mark.parametrize("freq", [[1.0] * 31, [], (ctypes.c_float * 31)(), (ctypes.c_double * 32)(), (ctypes.c_int * 64)()])
def test_frequencies_that_do_not_fit(lib, freq):
    """The library reads rot_dim / 2 fp32 values from the host array it is given."""
    with pytest.raises(ValueError):
        append(inv_freq=freq)
    assert not lib.calls


def test_frequencies_that_fit(lib):
    append(inv_freq=(ctypes.c_float * 32)())
    append(inv_freq=(ctypes.c_float * 40)())
    append(inv_freq=range(32))
    append(inv_freq=None, rot_dim=0)
    append(inv_freq=[], rot_dim=0)
    assert len(lib.calls) == 5
