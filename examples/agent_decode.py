"""Agents decoding over a shared pool, each with pages of its own.

A shared document is encoded once into a SharedKVPool; every agent then
generates tokens.  One decode step of a layer, for all agents:

    kvpages_append   the new tokens' queries and keys normed per head and turned to
                     their positions, keys and values quantised into the agents' pages
    kvpool_attend    the queries over the shared pool (out, lse)
    kvpages_attend   the queries over each agent's own pages, joined with the former

    python examples/agent_decode.py [--agents 15] [--pool-tokens 4096] [--steps 32] [--format k8v8] [--check]

Queries, keys and values are random (there is no model here); --check compares
every step with dense attention over the decoded caches.
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

FORMATS = {"bf16": kv.KVP_PAGES_BF16, "k8v8": kv.KVP_PAGES_K8V8, "k8v4": kv.KVP_PAGES_K8V4}


class AgentPages:
    """The agents' page container, its free list and tables (host bookkeeping)."""

    def __init__(self, agents, layers, kv_heads, dim, most_tokens, page_tokens, fmt):
        self.page = page_tokens
        self.max_pages = (most_tokens + page_tokens - 1) // page_tokens
        self.cfg = kv.PagesConfig(layers, kv_heads, dim, page_tokens, agents * self.max_pages, FORMATS[fmt])
        size = kv.kvpages_bytes(self.cfg)
        self.pages = torch.empty(size, dtype=torch.uint8, device="cuda")
        kv.check(kv.kvpages_init(self.cfg, self.pages, size, torch.cuda.current_stream()), "init")
        self.free = list(range(self.cfg.n_pages))
        self.table_host = torch.zeros(agents, self.max_pages, dtype=torch.int32)
        self.table = self.table_host.cuda()
        self.lens = torch.zeros(agents, dtype=torch.int32, device="cuda")
        self.held = 0  # tokens per agent (all agents step together here)

    def grow(self):
        """Room for one more token of every agent; their slots."""
        if self.held % self.page == 0:
            for a in range(self.table_host.shape[0]):
                self.table_host[a, self.held // self.page] = self.free.pop()
            self.table.copy_(self.table_host)
        slots = self.table[:, self.held // self.page].long() * self.page + self.held % self.page
        self.held += 1
        self.lens.fill_(self.held)
        return slots


def dense(q, ks, vs, scale):
    """Attention in fp32 over lists of [heads, tokens, dim] caches, query heads grouped."""
    outs = []
    for x, k, v in zip(q.float(), ks, vs):
        h = k.shape[0]
        s = torch.einsum("hgd,htd->hgt", x.view(h, -1, x.shape[-1]), k) * scale
        outs.append(torch.einsum("hgt,htd->hgd", torch.softmax(s, -1), v).reshape(x.shape))
    return torch.stack(outs)


def run(agents=15, layers=2, heads=32, kv_heads=8, dim=128, pool_tokens=4096, steps=32, page_tokens=16, fmt="k8v8",
        check=False, seed=0):
    """Runs `steps` decode steps; returns the largest error against dense
    attention relative to the largest value (check) and the time of a layer's step in us."""
    st = torch.cuda.current_stream()
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (layers, kv_heads, dim, pool_tokens)
    ks, vs = synth.kv_layers(layers, kv_heads, pool_tokens, dim, seed=seed, device="cuda")
    pool = torch.empty(kv.kvpool_pool_bytes(shape), dtype=torch.uint8, device="cuda")
    ws = torch.empty(kv.kvpool_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    kv.check(kv.kvpool_encode(shape, ks, vs, pool, pool.numel(), ws, ws.numel(), st), "encode")

    own = AgentPages(agents, layers, kv_heads, dim, steps, page_tokens, fmt)
    # rotary frequencies, laid out once
    freq = (ctypes.c_float * (dim // 2))(*[500000.0 ** (-2.0 * i / dim) for i in range(dim // 2)])
    norms = [(0.5 + torch.rand(dim, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]
    scale = 1.0 / math.sqrt(dim)
    q = torch.empty(agents, heads, dim, dtype=torch.bfloat16, device="cuda")
    pool_out = torch.empty(agents, heads, dim, device="cuda")
    pool_lse = torch.empty(agents, heads, device="cuda")
    out = torch.empty(agents, 1, heads, dim, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(agents, 1, heads, device="cuda")
    pool_ws = torch.empty(kv.kvpool_attend_workspace_bytes(shape, agents, heads), dtype=torch.uint8, device="cuda")
    own_ws = torch.empty(kv.kvpages_attend_workspace_bytes(own.cfg, agents, 1, heads), dtype=torch.uint8, device="cuda")

    worst, spent = 0.0, 0.0
    for step in range(steps):
        slots = own.grow()
        positions = torch.full((agents,), pool_tokens + step, dtype=torch.int64, device="cuda")
        for layer in range(layers):
            qkv = torch.randn(agents, heads + 2 * kv_heads, dim, generator=g, device="cuda").to(torch.bfloat16)
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            kv.check(kv.kvpages_append(own.pages, own.cfg, layer, agents, heads, qkv[:, :heads],
                                       qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:], slots, positions,
                                       norms[0], norms[1], 1e-5, dim, freq, q, None, None, st), "append")
            kv.check(kv.kvpool_attend(pool, shape, layer, agents, heads, q, scale, pool_out, pool_lse, pool_ws,
                                      pool_ws.numel(), st), "pool attention")
            kv.check(kv.kvpages_attend(own.pages, own.cfg, layer, agents, 1, heads, q, scale, own.table, own.max_pages,
                                       own.lens, pool_out, pool_lse, out, lse, own_ws, own_ws.numel(), st), "pages attention")
            b.record()
            if check:
                pk, pv = (torch.empty(kv_heads, pool_tokens, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
                none = [None] * layers
                kv.check(kv.kvpool_decode_into(pool, shape, layer, layer + 1, 1, none[:layer] + [pk] + none[layer + 1:],
                                               none[:layer] + [pv] + none[layer + 1:], st), "decode")
                ok, ov = (torch.empty(agents, kv_heads, own.held, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
                kv.check(kv.kvpages_read(own.pages, own.cfg, layer, agents, own.table, own.max_pages, own.lens, own.held, ok,
                                         ov, st), "read")
                ref = dense(q, [torch.cat([pk, x], 1).float() for x in ok], [torch.cat([pv, x], 1).float() for x in ov], scale)
                worst = max(worst, float((out[:, 0].float() - ref).abs().max() / pv.float().abs().max()))
            torch.cuda.synchronize()
            spent += a.elapsed_time(b) if step else 0.0
    kv.check(kv.kvpool_status(pool, st), "pool status")
    kv.check(kv.kvpages_status(own.pages, st), "pages status")
    return worst, spent * 1e3 / max(1, (steps - 1) * layers)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--agents", type=int, default=15)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--pool-tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--page-tokens", type=int, default=16)
    ap.add_argument("--format", choices=sorted(FORMATS), default="k8v8")
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args()
    kvbuild.build()
    worst, us = run(agents=a.agents, layers=a.layers, pool_tokens=a.pool_tokens, steps=a.steps,
                    page_tokens=a.page_tokens, fmt=a.format, check=a.check)
    print("%d agents over a pool of %d tokens, %d steps: %.1f us per layer and step%s" % (
        a.agents, a.pool_tokens, a.steps, us, "; largest error %.2g of the largest value" % worst if a.check else ""))
    return 0 if worst < 0.02 else 1


if __name__ == "__main__":
    sys.exit(main())
