"""An agent's long life over a shared pool: a prompt with a picture, then decode
steps that look at a window, its own cache held in 4 bits.

A shared document is encoded once into a SharedKVPool.  Of one layer, per agent:

    kvpages_append_axes    the prompt's queries and keys turned to positions of three axes,
                           keys and values quantised into the agent's 4-bit pages
    kvpool_attend          the prompt's queries over the shared pool (out, lse)
    kvprompt_attend        the prompt's queries over the prompt itself, each a window and the
                           first tokens, joined with the former
    kvpages_attend_window  then a token at a time, over the pages, joined likewise

    python examples/agent_prompt.py [--agents 3] [--pool-tokens 4096] [--prompt 700] [--steps 8]
                                    [--window 256] [--sinks 4] [--check]

Queries, keys and values are random (there is no model here); --check compares with dense
attention over what the pages hold.
"""
import argparse
import ctypes
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import agent_shared_compressed_gb300 as kv  # noqa: E402
from agent_shared_compressed_gb300 import build as kvbuild  # noqa: E402
from agent_shared_compressed_gb300 import synth  # noqa: E402


def positions(first, count, picture, columns):
    """Places of `count` tokens from `first` on [3][count]: text, but for the tokens of `picture`
    (a range), which share their time and have a row and a column."""
    t = torch.arange(count, device="cuda")
    shown = (t >= picture.start) & (t < picture.stop)
    at = (t - picture.start).clamp(min=0)
    return torch.stack([first + torch.where(shown, picture.start, t), first + torch.where(shown, picture.start + at // columns, t),
                        first + torch.where(shown, picture.start + at % columns, t)])


def dense(q, k, v, place, window, sinks, scale, base_out, base_lse):
    """One query [heads][dim] in fp32 over [tokens][kv heads][dim], joined with the base."""
    h, d = k.shape[1:]
    t = torch.arange(k.shape[0], device="cuda")
    see = (t <= place) & ((t > place - window) | (t < sinks))
    s = torch.einsum("hgd,thd->hgt", q.view(h, -1, d), k) * scale
    s = torch.where(see, s, -math.inf)
    lse = torch.logsumexp(s, -1).view(-1)
    out = torch.einsum("hgt,thd->hgd", torch.softmax(s, -1), v).reshape(-1, d)
    both = torch.logaddexp(lse, base_lse)
    return torch.exp(lse - both)[:, None] * out + torch.exp(base_lse - both)[:, None] * base_out


def run(agents=3, heads=32, kv_heads=8, dim=128, pool_tokens=4096, prompt=700, steps=8, window=256, sinks=4, page=16,
        check=False, seed=0):
    """The largest error against dense attention relative to the largest value (check)."""
    st = torch.cuda.current_stream()
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf16, f32, i32 = (dict(dtype=t, device="cuda") for t in (torch.bfloat16, torch.float32, torch.int32))
    shape = (1, kv_heads, dim, pool_tokens)
    ks, vs = synth.kv_layers(1, kv_heads, pool_tokens, dim, seed=seed, device="cuda")
    pool = torch.empty(kv.kvpool_pool_bytes(shape), dtype=torch.uint8, device="cuda")
    ws = torch.empty(kv.kvpool_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    kv.check(kv.kvpool_encode(shape, ks, vs, pool, pool.numel(), ws, ws.numel(), st), "encode")

    most = (prompt + steps + page - 1) // page
    cfg = kv.PagesConfig(1, kv_heads, dim, page, agents * most, kv.KVP_PAGES_K4V4)
    pages = torch.empty(kv.kvpages_bytes(cfg), dtype=torch.uint8, device="cuda")
    kv.check(kv.kvpages_init(cfg, pages, pages.numel(), st), "init")
    table = torch.arange(agents * most, **i32).view(agents, most)
    freq = (ctypes.c_float * (dim // 2))(*[500000.0 ** (-2.0 * i / dim) for i in range(dim // 2)])
    axes = (ctypes.c_uint8 * (dim // 2))(*[i % 3 for i in range(dim // 2)])
    scale = 1.0 / math.sqrt(dim)

    def slots(a, t):
        return (table[a, t // page].long() * page + t % page)

    def over_pool(q):
        """The queries [n][heads][dim] over the pool: every token is an agent of its own there."""
        n = q.shape[0]
        out, lse = torch.empty(n, heads, dim, **f32), torch.empty(n, heads, **f32)
        w = torch.empty(kv.kvpool_attend_workspace_bytes(shape, n, heads), dtype=torch.uint8, device="cuda")
        kv.check(kv.kvpool_attend(pool, shape, 0, n, heads, q, scale, out, lse, w, w.numel(), st), "pool attention")
        return out, lse

    def write(x, slot, pos, outs):
        n = x.shape[0]
        q = torch.empty(n, heads, dim, **bf16)
        k, v = (torch.empty(n, kv_heads, dim, **bf16) if outs else None for _ in range(2))
        kv.check(kv.kvpages_append_axes(pages, cfg, 0, n, heads, x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:],
                                        slot, pos, 3, axes, None, None, 0.0, dim, freq, q, k, v, st), "append")
        return q, k, v

    # the prompts, agent after agent
    n = agents * prompt
    x = torch.randn(n, heads + 2 * kv_heads, dim, generator=g, device="cuda").to(torch.bfloat16)
    t = torch.arange(prompt, device="cuda")
    slot = torch.cat([slots(a, t) for a in range(agents)])
    pos = positions(pool_tokens, prompt, range(10, 10 + min(prompt - 10, 31 * 8)) if prompt > 10 else range(0), 31)
    q, k, v = write(x, slot, pos.repeat(1, agents).contiguous(), True)
    base = over_pool(q)
    first = torch.arange(agents + 1, **i32) * prompt
    pshape = kv.PromptShape(agents, n, n, heads, kv_heads, dim)
    pws = torch.empty(kv.kvprompt_workspace_bytes(pshape), dtype=torch.uint8, device="cuda")
    error = torch.zeros(1, **i32)
    out = torch.empty(n, heads, dim, **bf16)
    kv.check(kv.kvprompt_attend(pshape, q, k, v, first, first[:-1], torch.full((agents,), prompt, **i32), scale, window, sinks,
                                *base, out, None, error, pws, pws.numel(), st), "prompt attention")
    kv.check(kv.kvprompt_status(error, st), "prompt status")
    worst = 0.0
    if check:
        for a in range(agents):
            own = slice(a * prompt, (a + 1) * prompt)
            for i in sorted({0, 1, prompt // 3, prompt - 1}):
                at = a * prompt + i
                ref = dense(q[at].float(), k[own].float(), v[own].float(), i, window, sinks, scale, base[0][at], base[1][at])
                worst = max(worst, float((out[at].float() - ref).abs().max() / v.float().abs().max()))

    # then a token at a time
    aws = torch.empty(kv.kvpages_attend_workspace_bytes(cfg, agents, 1, heads), dtype=torch.uint8, device="cuda")
    for step in range(steps):
        place = prompt + step
        x = torch.randn(agents, heads + 2 * kv_heads, dim, generator=g, device="cuda").to(torch.bfloat16)
        here = torch.full((1,), place, dtype=torch.int64, device="cuda")
        q, _, _ = write(x, torch.cat([slots(a, here) for a in range(agents)]),
                        torch.full((3, agents), pool_tokens + place, dtype=torch.int64, device="cuda"), False)
        base = over_pool(q)
        lens = torch.full((agents,), place + 1, **i32)
        out = torch.empty(agents, 1, heads, dim, **bf16)
        kv.check(kv.kvpages_attend_window(pages, cfg, 0, agents, 1, heads, q, scale, window, sinks, table, most, lens, *base, out,
                                          None, aws, aws.numel(), st), "pages attention")
        if check:
            pk, pv = (torch.empty(agents, kv_heads, place + 1, dim, **bf16) for _ in range(2))
            kv.check(kv.kvpages_read(pages, cfg, 0, agents, table, most, lens, place + 1, pk, pv, st), "read")
            for a in range(agents):
                ref = dense(q[a].float(), pk[a].float().transpose(0, 1), pv[a].float().transpose(0, 1), place, window, sinks, scale,
                            base[0][a], base[1][a])
                worst = max(worst, float((out[a, 0].float() - ref).abs().max() / pv.float().abs().max()))
    kv.check(kv.kvpool_status(pool, st), "pool status")
    kv.check(kv.kvpages_status(pages, st), "pages status")
    return worst


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("agents", 3), ("pool-tokens", 4096), ("prompt", 700), ("steps", 8), ("window", 256), ("sinks", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args()
    kvbuild.build()
    worst = run(agents=a.agents, pool_tokens=a.pool_tokens, prompt=a.prompt, steps=a.steps, window=a.window, sinks=a.sinks,
                check=a.check)
    print("%d agents over a pool of %d tokens: prompts of %d, %d steps%s" % (
        a.agents, a.pool_tokens, a.prompt, a.steps, "; largest error %.2g of the largest value" % worst if a.check else ""))
    return 0 if worst < 0.02 else 1


if __name__ == "__main__":
    sys.exit(main())
