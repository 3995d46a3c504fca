"""GPU tests of attention over pages where it can go wrong: bounded waits that
run out for some lanes only."""
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
