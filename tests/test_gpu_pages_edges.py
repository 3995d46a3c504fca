"""GPU tests of attention over pages where it can go wrong: bounded waits that
run out for some lanes only, joins in place."""
import numpy as np
import pytest
import torch

import agent_shared_compressed_gb300 as kv
from agent_shared_compressed_gb300 import build as kvbuild
import pageshelp as P
from test_gpu_pages import FMTS, Pages, _check_attend, _f64, _kv, _split

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    kvbuild.build()
    kv.load()


# --- waits ------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lanes", [0x1, 0x80000000, 0x00010000, 0xAAAAAAAA])
@pytest.mark.parametrize("roomy", [False, True])
def test_wait_that_runs_out_for_some_lanes(fmt, lanes, roomy):
    """A wait that some lanes give up and others do not ends the warp's run as a
    whole, in either split of the work; the call after it is right."""
    H, d, lens = 4, 128, [900, 20, 0]
    k, v = _kv(sum(lens), H, d, 30)
    pg = Pages(fmt, H, d, 64, lens, max_pages=4096 if roomy else None)
    pg.append(k, v)
    q = torch.randn(3, 1, 8, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    assert kv.kvp_test_limit_next_pages_attend_lanes(0, lanes) == kv.KVP_OK
    pg.attend(q, 0.1)
    assert pg.status() == kv.KVP_ERR_TIMEOUT
    assert kv.kvpages_init(pg.cfg, pg.buf.t, pg.buf.nbytes) == kv.KVP_OK  # clears the error word; the pages stay
    out, lse = pg.attend(q, 0.1)
    assert pg.status() == kv.KVP_OK
    _check_attend(out, lse, _f64(q), _split(P.held(_f64(k), fmt, False), lens), _split(P.held(_f64(v), fmt, True), lens),
                  lens, 0.1)


# --- joins -------------------------------------------------------------------------

JOINS = [  # H, d, page, lens, m, query heads, table width: which part of the code ends a row
    (4, 128, 16, [40, 0, 7, 64], 1, 16, None),       # teams' merges and whole tiles, tiles of 4
    (4, 64, 16, [150, 3, 0], 3, 8, None),            # of 8
    (2, 128, 16, [90, 33], 8, 8, None),              # of 16
    (4, 128, 16, [4000, 0, 2500], 1, 16, 4096),      # cut from the list, joined
    (2, 64, 16, [3000, 900], 3, 8, 4096),
    (8, 128, 16, [20] * 300, 1, 32, 4096),           # many whole tiles of the list
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", JOINS)
def test_join_with_lse_in_place(fmt, case):
    """lse written over base_lse gives what another tensor for it gives, bit for bit."""
    H, d, page, lens, m, nq, width = case
    pg = Pages(fmt, H, d, page, lens, max_pages=width)
    k, v = _kv(sum(lens), H, d, 31)
    pg.append(k, v, outs=False)
    g = torch.Generator().manual_seed(2)
    q = torch.randn(len(lens), m, nq, d, generator=g).to(torch.bfloat16).cuda()
    bo, bl = torch.randn(q.shape, generator=g).cuda(), (torch.randn(q.shape[:3], generator=g) * 3).cuda()
    out, lse = pg.attend(q, 0.1, bo, bl)
    wsb = kv.kvpages_attend_workspace_bytes(pg.cfg, len(lens), m, nq)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    for _ in range(5):
        o, both = torch.empty_like(q), bl.clone()
        assert kv.kvpages_attend(pg.buf.t, pg.cfg, 0, len(lens), m, nq, q, 0.1, pg.table_d, pg.max_pages, pg.lens_d, bo,
                                 both, o, both, ws, wsb) == kv.KVP_OK
        torch.cuda.synchronize()
        assert np.array_equal(_f64(o), out) and np.array_equal(both.cpu().numpy().astype(np.float64), lse)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("width", [None, 4096])
def test_base_that_is_not_a_number(fmt, width):
    """A base whose lse is NaN gives NaN, also for queries that see no token of
    their own; one whose lse is -inf gives what there is, whatever it holds."""
    H, nq, d, lens = 2, 4, 64, [0, 40, 0, 40]
    pg = Pages(fmt, H, d, 16, lens, max_pages=width)
    k, v = _kv(sum(lens), H, d, 32)
    pg.append(k, v, outs=False)
    q = torch.randn(4, 1, nq, d, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    bo, bl = torch.full(q.shape, float("nan"), device="cuda"), torch.full(q.shape[:3], float("nan"), device="cuda")
    bl[2:] = -float("inf")
    out, lse = pg.attend(q, 0.1, bo, bl)
    alone = pg.attend(q, 0.1)
    assert np.all(np.isnan(lse[:2])) and np.all(np.isnan(out[:2]))
    assert np.array_equal(lse[2:], alone[1][2:]) and np.array_equal(out[2:], alone[0][2:])
