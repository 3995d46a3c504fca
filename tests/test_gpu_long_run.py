"""GPU tests of the operators for long-lived agents as they are used together: a prompt
written with several axes, attended over with the pool, continued a token at a time; and
the example that does so."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import agent_shared_compressed_gb300 as kv
from agent_shared_compressed_gb300 import build as kvbuild
from agent_shared_compressed_gb300 import synth
import longhelp as Lg
import pageshelp as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    kvbuild.build()
    kv.load()


@pytest.mark.parametrize("fmt", ["bf16", "k4v4"])
@pytest.mark.parametrize("d,window,sinks", [(128, 40, 3), (64, 0, 0)])
def test_a_prompt_is_what_its_tokens_one_by_one_are(fmt, d, window, sinks):
    """Two sequences, written as prompts, attended by kvprompt_attend over what the pages hold
    (k_out, v_out), then the same tokens by kvpages_attend_window, eight at a time, over the pages:
    both against 64 bits with the pool joined in, all in one graph on another stream.  What pages
    of 4 bits hold reaches the prompt's attention rounded to bf16, the pages' own exactly."""
    H, nq, T, lens = 2, 8, 96, [75, 33]
    rng = np.random.default_rng(d + window)
    n = sum(lens)
    ks, vs = synth.kv_layers(1, H, T, d, seed=3, device="cuda")
    shape = (1, H, d, T)
    pool = torch.empty(kv.kvpool_pool_bytes(shape), dtype=torch.uint8, device="cuda")
    ws = torch.empty(kv.kvpool_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    kv.check(kv.kvpool_encode(shape, ks, vs, pool, pool.numel(), ws, ws.numel()))
    pg = Lg.Pages(fmt, H, d, 16, lens, seed=1)
    x = Lg.bf16(rng.standard_normal((n, nq + 2 * H, d))).cuda()
    pos = torch.from_numpy(rng.integers(0, 5000, (3, n))).cuda()
    freq = [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]
    axes = [i * 3 // (d // 2) for i in range(d // 2)]
    bf, f32, i32 = (dict(dtype=t, device="cuda") for t in (torch.bfloat16, torch.float32, torch.int32))
    q, k, v, out = (torch.empty(n, h, d, **bf) for h in (nq, H, H, nq))
    bo, bl, lse = torch.empty(n, nq, d, **f32), torch.empty(n, nq, **f32), torch.empty(n, nq, **f32)
    pws = torch.empty(kv.kvpool_attend_workspace_bytes(shape, n, nq), dtype=torch.uint8, device="cuda")
    qf = torch.tensor([0, lens[0], n], **i32)
    pshape = kv.PromptShape(2, n, n, nq, H, d)
    aws = torch.empty(kv.kvprompt_workspace_bytes(pshape), dtype=torch.uint8, device="cuda")
    error = torch.zeros(1, **i32)
    scale = 1 / math.sqrt(d)
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        c = torch.cuda.current_stream()
        kv.check(kv.kvpages_append_axes(pg.buf.t, pg.cfg, 0, n, nq, x[:, :nq], x[:, nq:nq + H], x[:, nq + H:], pg.slots, pos, 3, axes,
                                        None, None, 0.0, d, freq, q, k, v, c))
        kv.check(kv.kvpool_attend(pool, shape, 0, n, nq, q, scale, bo, bl, pws, pws.numel(), c))
        kv.check(kv.kvprompt_attend(pshape, q, k, v, qf, qf[:2], pg.lens_d, scale, window, sinks, bo, bl, out, lse, error, aws,
                                    aws.numel(), c))
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
    assert kv.kvprompt_status(error) == kv.KVP_OK and pg.status() == kv.KVP_OK and kv.kvpool_status(pool) == kv.KVP_OK
    hq, hk, hv, ho, hl = (Lg.f64(t) for t in (q, k, v, out, lse))
    hbo, hbl = bo.cpu().numpy().astype(np.float64), bl.cpu().numpy().astype(np.float64)
    for b, m in enumerate(lens):
        i = slice(sum(lens[:b]), sum(lens[:b + 1]))
        ro, rl, mass, reach = Lg.prompt(hq[i], hk[i], hv[i], 0, window, sinks, scale)
        ro, rl, mass = Lg.join(ro, rl, mass, hbo[i], hbl[i])
        Lg.check(ho[i], hl[i], ro, rl, mass, reach, 2.0 ** -8)
        prompt = (ro, mass, reach)
        # the last eight tokens again, over the pages
        last = slice(i.stop - 8, i.stop)
        lens_d = torch.zeros(2, **i32)
        lens_d[b] = m
        pg.lens_d, q8 = lens_d, torch.zeros(2, 8, nq, d, **bf)
        q8[b] = q[last]
        b8o, b8l = torch.zeros(2, 8, nq, d, **f32), torch.zeros(2, 8, nq, **f32)
        b8o[b], b8l[b] = bo[last], bl[last]
        o8, _ = pg.attend(q8, scale, window, sinks, b8o, b8l)
        # held values are off by a bf16 rounding in the prompt's own: 2^-8 of a key moves a score by
        # 2^-8 of its reach, and 2^-8 of a value; of the 16-bit pages' nothing
        off = (0.0 if fmt == "bf16" else 2.0 ** -8) * (1 + 2 * prompt[2][-8:, :, None]) + 2.0 ** -8 + 2.0 ** -14
        assert np.all(np.abs(o8[b] - prompt[0][-8:]) <= 2.0 ** -8 * np.abs(prompt[0][-8:]) + off * prompt[1][-8:])


@pytest.mark.parametrize("more", [dict(), dict(prompt=9, window=5, sinks=0, steps=2, agents=1), dict(dim=64, kv_heads=2, heads=6, prompt=300)])
def test_example_agent_prompt(more):
    """The example runs, and its own comparison with dense attention holds: values, weights and the
    output round to 2^-8 each, the steps' keys that are read back in bf16 move a score by up to 2^-8 of
    sum |q k| (below 1 where weights matter): five times 2^-8 of the largest value."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "agent_prompt.py")
    spec = importlib.util.spec_from_file_location("agent_prompt", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert mod.run(**{**dict(pool_tokens=512, steps=3, check=True), **more}) < 0.02
