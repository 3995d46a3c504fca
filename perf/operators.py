"""The paged agent-cache operators as measured workloads.

An agent reads the shared pool and keeps its own tokens in pages.  Four kinds
of pass, by a case's "op":

* write:  new tokens' queries, keys and values (as the model's fused
          projection leaves them) -> per-head norm, position rotation,
          quantised write into the pages; returns the queries and the keys and
          values as the cache now holds them (a prompt's own attention takes
          these).
* read:   the pages' tokens back as bf16 past_key_values.
* attend: attention of each sequence's newest tokens over its pages, joined
          with attention over the pool where "join" is set.
* step:   one decode step of a layer: write one token per sequence, attend.

With `own` false everything is elementary torch arithmetic in 32 bits on plain
paged tensors (64 bits for the rotation's angles and for the 4-bit codes,
whose values lie next to a border); with `own` true it is the library's calls
on its own page container.
"""
import math

import torch

own = False

EPS = 1e-5
THETA = 500000.0
GROUP = 32


# --- cases -------------------------------------------------------------------

def _case(name, op, fmt, heads, kv_heads, dim, page, seqs, len_min, len_max, q_tokens=1, norm=False, join=False):
    c = dict(op=op, fmt=fmt, heads=heads, kv_heads=kv_heads, dim=dim, page=page, seqs=seqs, len_min=len_min,
             len_max=len_max, q_tokens=q_tokens, norm=norm, join=join)
    return dict(c, name=name) if name else c


def listed():
    return [
        # 15 agents each write the token they have just produced: latency
        _case("write-15-tokens", "write", "k8v8", 32, 8, 128, 16, 15, 1, 1, norm=True),
        # an agent's long private prompt
        _case("write-prompt-8k", "write", "k8v4", 32, 8, 128, 64, 1, 8192, 8192, norm=True),
        # three agents' ragged prompts on a model without grouped heads, cache kept in 16 bits
        _case("write-ragged-d64", "write", "bf16", 32, 32, 64, 32, 3, 37, 1851),
        # 15 agents' caches handed to code that wants past_key_values
        _case("read-4k-15agents", "read", "k8v8", 32, 8, 128, 64, 15, 4096, 4096),
        # a ragged handful, lengths from none
        _case("read-ragged-d64", "read", "k8v4", 32, 32, 64, 32, 7, 0, 1851),
        # one decode step of a layer: short private tails beside the pool
        _case("step-15agents", "step", "k8v8", 32, 8, 128, 16, 15, 1, 513, norm=True, join=True),
        # attention over 15 private 4K caches kept in 16 bits
        _case("attend-4k-bf16", "attend", "bf16", 32, 8, 128, 64, 15, 4096, 4096),
        # attention over four 32K caches
        _case("attend-32k", "attend", "k8v8", 32, 8, 128, 64, 4, 32768, 32768),
        # many ragged sequences, one query head per KV head, some of them empty
        _case("attend-ragged-d64", "attend", "k8v4", 32, 32, 64, 32, 64, 0, 1851),
        # five drafted tokens each, checked at once, joined with the pool
        _case("attend-drafts", "attend", "k8v4", 32, 8, 128, 16, 8, 700, 4096, q_tokens=5, join=True),
        # a single long sequence: nothing but the length to split over
        _case("attend-one-128k", "attend", "k8v4", 32, 8, 128, 128, 1, 131072, 131072),
    ]


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "step"])
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 16, 32])
    group = rng.choice([1, 2, 3, 4, 5, 8]) if kv_heads <= 8 else 1
    q_tokens = rng.choice([1, 1, 1, 2, 5, 8]) if op == "attend" else 1
    seqs = int(2 ** rng.uniform(0, 6.5))
    most = {"write": 8192 * 8 * 128, "read": 30000 * 8 * 128}.get(op, 60000 * 8 * 128 // max(1, q_tokens * group // 8))
    top = max(1, min(131072, most // (seqs * kv_heads * dim)))
    len_max = max(1, int(2 ** rng.uniform(0, math.log2(top))))
    len_min = rng.choice([0, 1, len_max // 3, len_max])
    return _case(None, op, rng.choice(["bf16", "k8v8", "k8v4"]), kv_heads * group, kv_heads, dim,
                 rng.choice([16, 32, 64, 128]), seqs, min(len_min, len_max), len_max, q_tokens,
                 op in ("write", "step") and rng.random() < 0.5, op in ("attend", "step") and rng.random() < 0.5)


def _lengths(case):
    """Lengths spread over the case's range; the first is the longest."""
    lo, hi, n = case["len_min"], case["len_max"], case["seqs"]
    at_least = 1 if case["op"] == "step" else 0
    return [max(at_least, hi - int((hi - lo) * ((i * 0.6180339887498949) % 1.0) + (0.5 if i else 0))) for i in range(n)]


def _pair_bytes(case):
    """Bytes that one cached token of one KV head takes, keys and values."""
    d = case["dim"]
    return {"bf16": 4 * d, "k8v8": 2 * d + 4 * (d // GROUP), "k8v4": d + d // 2 + 6 * (d // GROUP)}[case["fmt"]]


def work(case):
    nq, h, d, b, m = case["heads"], case["kv_heads"], case["dim"], case["seqs"], case["q_tokens"]
    lens, c = _lengths(case), _pair_bytes(case)
    total, nbytes, flops = sum(lens), 0, 0
    if case["op"] in ("write", "step"):
        n = total if case["op"] == "write" else b
        nbytes += n * (nq + 2 * h) * d * 2 + n * nq * d * 2 + n * h * c + n * 16
        nbytes += n * h * d * 4 if case["op"] == "write" else 0
        flops += n * (nq + 2 * h) * d * 10
    if case["op"] == "read":
        nbytes += total * h * c + b * h * max(lens) * d * 4
        flops += total * h * d * 4
    if case["op"] in ("attend", "step"):
        nbytes += total * h * c + b * m * nq * (2 * d + 2 * d + 4) + (b * m * nq * (4 * d + 4) if case["join"] else 0)
        flops += 4 * total * m * nq * d
    return {"bytes": nbytes, "flops": flops}


# --- inputs --------------------------------------------------------------------

_FORMATS = {"bf16": "KVP_PAGES_BF16", "k8v8": "KVP_PAGES_K8V8", "k8v4": "KVP_PAGES_K8V4"}


def _keys(n, h, d, g):
    """Keys with a few strong channels per head."""
    k = torch.randn(n, h, d, generator=g, device="cuda")
    strong = torch.rand(h, d, generator=g, device="cuda").argsort(dim=1)[:, :4]
    return (k * torch.ones(h, d, device="cuda").scatter_(1, strong, 20.0)).to(torch.bfloat16)


def _values(n, h, d, g):
    """Heavier tails than a Gaussian's (Student's t, 5 degrees)."""
    z = torch.randn(n, h, d, generator=g, device="cuda")
    w = torch.randn(5, n, h, d, generator=g, device="cuda").square().sum(0)
    return (0.5 * z / torch.sqrt(w / 5)).to(torch.bfloat16)


def _inputs(case, seed):
    """What a model and its scheduler have in hand, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    nq, h, d, p, b, m = (case[k] for k in ("heads", "kv_heads", "dim", "page", "seqs", "q_tokens"))
    lens = _lengths(case)
    per_seq = [(n + p - 1) // p for n in lens]
    max_pages = max(1, max(per_seq))
    n_pages = sum(per_seq) + 3
    free = torch.randperm(n_pages, generator=g, device="cuda")
    table = torch.zeros(b, max_pages, dtype=torch.int32, device="cuda")
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    held = torch.arange(max_pages, device="cuda")[None, :] < ((lens_t + p - 1) // p)[:, None]
    table[held] = free[: sum(per_seq)].to(torch.int32)
    seq = torch.repeat_interleave(torch.arange(b, device="cuda"), lens_t.long())
    index = torch.arange(sum(lens), device="cuda") - (torch.cumsum(lens_t.long(), 0) - lens_t.long())[seq]
    slots = table[seq, index // p].long() * p + index % p
    s = dict(lens=lens_t, table=table, max_pages=max_pages, n_pages=n_pages, max_len=max(lens))
    first = 4096 + int(torch.randint(0, 1000, (1,), generator=g, device="cuda"))  # the pool's tokens come before
    if case["op"] != "write":
        s["old_k"], s["old_v"], s["old_slots"] = _keys(sum(lens), h, d, g), _values(sum(lens), h, d, g), slots
    if case["op"] in ("write", "step"):
        if case["op"] == "step":
            last = (torch.cumsum(lens_t.long(), 0) - 1)
            slots, index = slots[last], index[last]
        n = slots.numel()
        s["new"] = torch.cat([torch.randn(n, nq, d, generator=g, device="cuda").to(torch.bfloat16), _keys(n, h, d, g),
                              _values(n, h, d, g)], dim=1)  # one row per token, as the fused projection writes it
        s["slots"], s["positions"] = slots, first + index
        if case["norm"]:
            s["q_norm"] = (0.5 + torch.rand(d, generator=g, device="cuda")).to(torch.bfloat16)
            s["k_norm"] = (0.5 + torch.rand(d, generator=g, device="cuda")).to(torch.bfloat16)
    if case["op"] == "attend":
        s["q"] = torch.randn(b, m, nq, d, generator=g, device="cuda").to(torch.bfloat16)
    if case["join"]:
        s["base_out"] = 0.1 * torch.randn(b, m, nq, d, generator=g, device="cuda")
        s["base_lse"] = 5.0 + torch.rand(b, m, nq, generator=g, device="cuda") * 3
    return s


def _inv_freq(d):
    return [THETA ** (-2.0 * i / d) for i in range(d // 2)]


def prepare(case, seed):
    s = _inputs(case, seed)
    nq, h, d, p, b, m = (case[k] for k in ("heads", "kv_heads", "dim", "page", "seqs", "q_tokens"))
    s["case"] = case
    s["scale"] = 1.0 / math.sqrt(d)
    if own:
        _prepare_own(s)
    else:
        n = s["n_pages"] * p
        s["freq"] = torch.tensor(_inv_freq(d), dtype=torch.float32, device="cuda")
        if case["fmt"] == "bf16":
            s["kc"], s["vc"] = (torch.zeros(n, h, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        else:
            s["kc"] = torch.zeros(n, h, d, dtype=torch.int8, device="cuda")
            s["ks"] = torch.zeros(n, h, d // GROUP, dtype=torch.float16, device="cuda")
            s["vc"], s["vs"] = torch.zeros_like(s["kc"]), torch.zeros_like(s["ks"])
            if case["fmt"] == "k8v4":
                s["vz"] = torch.zeros_like(s["ks"])
        if "old_k" in s:
            _store(s, s["old_slots"], s["old_k"].float(), s["old_v"].float())
    for k in ("old_k", "old_v", "old_slots"):
        s.pop(k, None)
    return s


# --- the plain forms -------------------------------------------------------------

def _code8(x):
    """8-bit codes of groups of 32 and their scales."""
    x = x.unflatten(-1, (-1, GROUP))
    s = (x.abs().amax(-1) * (1.0 / 127.0)).to(torch.float16)
    sf = s.float()[..., None]
    code = torch.where(sf > 0, torch.round(x / torch.where(sf > 0, sf, 1.0)), 0.0).clamp(-127, 127)
    return code.flatten(-2).to(torch.int8), s


def _code4(x):
    """4-bit codes of groups of 32, their scales and zero points."""
    x = x.unflatten(-1, (-1, GROUP))
    lo, hi = x.amin(-1), x.amax(-1)
    s = ((hi - lo) * (1.0 / 15.0)).to(torch.float16)
    z = lo.to(torch.float16)
    sd = s.double()[..., None]
    code = torch.where(sd > 0, torch.round((x.double() - z.double()[..., None]) / torch.where(sd > 0, sd, 1.0)), 0.0)
    return code.clamp(0, 15).flatten(-2).to(torch.int8), s, z


def _value(code, s, z=None):
    x = code.float().unflatten(-1, (-1, GROUP)) * s.float()[..., None]
    return (x if z is None else x + z.float()[..., None]).flatten(-2)


def _store(s, slots, k, v):
    """Writes keys and values (32 bits) into the plain pages; the values that the pages then hold."""
    fmt = s["case"]["fmt"]
    if fmt == "bf16":
        s["kc"][slots], s["vc"][slots] = k.to(torch.bfloat16), v.to(torch.bfloat16)
        return k.to(torch.bfloat16), v.to(torch.bfloat16)
    kc, ks = _code8(k)
    s["kc"][slots], s["ks"][slots] = kc, ks
    if fmt == "k8v8":
        vc, vs = _code8(v)
        s["vc"][slots], s["vs"][slots] = vc, vs
        return _value(kc, ks).to(torch.bfloat16), _value(vc, vs).to(torch.bfloat16)
    vc, vs, vz = _code4(v)
    s["vc"][slots], s["vs"][slots], s["vz"][slots] = vc, vs, vz
    return _value(kc, ks).to(torch.bfloat16), _value(vc, vs, vz).to(torch.bfloat16)


def _load(s):
    """Every sequence's tokens [seqs, longest, heads, dim] in 32 bits (rows past a sequence's end: whatever its table holds)."""
    p = s["case"]["page"]
    t = torch.arange(max(1, s["max_len"]), device="cuda")
    at = s["table"].long()[:, t // p] * p + t % p
    fmt = s["case"]["fmt"]
    if fmt == "bf16":
        return s["kc"][at].float(), s["vc"][at].float()
    return (_value(s["kc"][at], s["ks"][at]),
            _value(s["vc"][at], s["vs"][at], s["vz"][at] if fmt == "k8v4" else None))


def _normed(x, w):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _turned(x, cos, sin):
    half = x.shape[-1] // 2
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _write(s):
    case = s["case"]
    nq, h = case["heads"], case["kv_heads"]
    x = s["new"].float()
    angle = s["positions"].double()[:, None] * s["freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q = _turned(_normed(x[:, :nq], s.get("q_norm")), cos, sin).to(torch.bfloat16)
    k = _turned(_normed(x[:, nq:nq + h], s.get("k_norm")), cos, sin)
    k, v = _store(s, s["slots"], k, x[:, nq + h:])
    return q, k, v


def _attend(s, q):
    case = s["case"]
    b, m, nq, d = q.shape
    h = case["kv_heads"]
    k, v = _load(s)
    x = torch.einsum("bmhgd,bthd->bhmgt", q.float().view(b, m, h, nq // h, d), k) * s["scale"]
    limit = s["lens"].long()[:, None] - torch.arange(m - 1, -1, -1, device="cuda")  # tokens that each query sees
    seen = torch.arange(k.shape[1], device="cuda")[None, None, :] < limit[:, :, None]
    x = torch.where(seen[:, None, :, None, :], x, -math.inf)
    v = torch.where((torch.arange(k.shape[1], device="cuda")[None, :] < s["lens"][:, None])[:, :, None, None], v, 0.0)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    w = torch.exp(x - top)
    total = w.sum(-1, keepdim=True)
    out = torch.einsum("bhmgt,bthd->bmhgd", w / torch.where(total > 0, total, 1.0), v).reshape(b, m, nq, d)
    lse = (top + torch.log(total))[..., 0].permute(0, 2, 1, 3).reshape(b, m, nq)
    if case["join"]:
        both = torch.maximum(lse, s["base_lse"])
        both = both + torch.log(torch.exp(lse - both) + torch.exp(s["base_lse"] - both))
        out = torch.exp(lse - both)[..., None] * out + torch.exp(s["base_lse"] - both)[..., None] * s["base_out"]
        lse = both
    return out.to(torch.bfloat16), lse


def _read(s):
    k, v = _load(s)
    there = (torch.arange(k.shape[1], device="cuda")[None, :] < s["lens"][:, None])[:, :, None, None]
    k, v = (torch.where(there, x, 0.0).to(torch.bfloat16).transpose(1, 2).contiguous() for x in (k, v))
    return {"k": k, "v": v}


# --- the library's calls ------------------------------------------------------------

def _prepare_own(s):
    import ctypes

    import agent_shared_compressed_gb300 as kv
    case = s["case"]
    nq, h, d, p, b, m = (case[k] for k in ("heads", "kv_heads", "dim", "page", "seqs", "q_tokens"))
    cfg = kv.PagesConfig(1, h, d, p, s["n_pages"], getattr(kv, _FORMATS[case["fmt"]]))
    size = kv.kvpages_bytes(cfg)
    pages = torch.empty(size, dtype=torch.uint8, device="cuda")
    kv.check(kv.kvpages_init(cfg, pages, size, _stream()), "init")
    s.update(kv=kv, cfg=cfg, pages=pages, freq=(ctypes.c_float * (d // 2))(*_inv_freq(d)))
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    if "old_k" in s and s["old_k"].shape[0]:
        kv.check(kv.kvpages_append(pages, cfg, 0, s["old_k"].shape[0], 0, None, s["old_k"], s["old_v"], s["old_slots"],
                                   None, None, None, 0.0, 0, None, None, None, None, _stream()), "append")
    if "new" in s:
        n = s["new"].shape[0]
        s["q_out"] = torch.empty(n, nq, d, **bf16)
        s["k_out"], s["v_out"] = ((torch.empty(n, h, d, **bf16) for _ in range(2)) if case["op"] == "write" else (None, None))
    if case["op"] == "read":
        s["k_out"], s["v_out"] = (torch.empty(b, h, max(1, s["max_len"]), d, **bf16) for _ in range(2))
    if case["op"] in ("attend", "step"):
        s["ws"] = torch.empty(kv.kvpages_attend_workspace_bytes(cfg, b, m, nq), dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty(b, m, nq, d, **bf16)
        s["lse"] = torch.empty(b, m, nq, dtype=torch.float32, device="cuda")


def _stream():
    return torch.cuda.current_stream()


def _own_write(s):
    kv, case, x = s["kv"], s["case"], s["new"]
    nq, h, d = case["heads"], case["kv_heads"], case["dim"]
    kv.check(kv.kvpages_append(s["pages"], s["cfg"], 0, x.shape[0], nq, x[:, :nq], x[:, nq:nq + h], x[:, nq + h:],
                               s["slots"], s["positions"], s.get("q_norm"), s.get("k_norm"), EPS, d, s["freq"],
                               s["q_out"], s["k_out"], s["v_out"], _stream()))


def _own_attend(s, q):
    kv, case = s["kv"], s["case"]
    kv.check(kv.kvpages_attend(s["pages"], s["cfg"], 0, case["seqs"], case["q_tokens"], case["heads"], q, s["scale"],
                               s["table"], s["max_pages"], s["lens"], s.get("base_out"), s.get("base_lse"), s["out"],
                               s["lse"], s["ws"], s["ws"].numel(), _stream()))
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    op = state["case"]["op"]
    if own:
        if op == "write":
            _own_write(state)
            return {"q": state["q_out"], "k": state["k_out"], "v": state["v_out"]}
        if op == "read":
            kv, case = state["kv"], state["case"]
            kv.check(kv.kvpages_read(state["pages"], state["cfg"], 0, case["seqs"], state["table"], state["max_pages"],
                                     state["lens"], max(1, state["max_len"]), state["k_out"], state["v_out"], _stream()))
            return {"k": state["k_out"], "v": state["v_out"]}
        if op == "step":
            _own_write(state)
            return _own_attend(state, state["q_out"])
        return _own_attend(state, state["q"])
    if op == "write":
        q, k, v = _write(state)
        return {"q": q, "k": k, "v": v}
    if op == "read":
        return _read(state)
    q = _write(state)[0][:, None] if op == "step" else state["q"]
    out, lse = _attend(state, q)
    return {"out": out, "lse": lse}


# --- the definition in 64 bits ---------------------------------------------------------

def _exact_groups(x, fmt, values):
    """What the cache holds for x (64 bits, [..., dim]), by the format's definition (16 bits: before their rounding)."""
    if fmt == "bf16":
        return x
    blocks = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    if values and fmt == "k8v4":
        low = blocks.min(-1, keepdim=True).values
        step = ((blocks.max(-1, keepdim=True).values - low) / 15).to(torch.float16).double()
        zero = low.to(torch.float16).double()
        n = ((blocks - zero) / step).round().clamp(0, 15)
        held = torch.where(step == 0, zero.expand_as(blocks), n * step + zero)
    else:
        step = (blocks.abs().max(-1, keepdim=True).values / 127).to(torch.float16).double()
        n = (blocks / step).round().clamp(-127, 127)
        held = torch.where(step == 0, torch.zeros_like(blocks), n * step)
    return held.reshape(x.shape)


def _exact_heads(x, weight, positions):
    """Norm and rotation of [tokens, heads, dim] in 64 bits: pairs (i, i + dim/2) as complex numbers."""
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
    d = x.shape[-1]
    freq = torch.tensor(_inv_freq(d), dtype=torch.float32).double().cuda()
    turn = torch.polar(torch.ones(positions.numel(), d // 2, dtype=torch.float64, device="cuda"),
                       positions.double()[:, None] * freq)
    y = torch.complex(x[..., : d // 2].contiguous(), x[..., d // 2:].contiguous()) * turn[:, None]
    return torch.cat([y.real, y.imag], -1)


def exact(case, seed):
    s = _inputs(case, seed)
    nq, h, d, b, m, fmt = (case[k] for k in ("heads", "kv_heads", "dim", "seqs", "q_tokens", "fmt"))
    if case["op"] in ("write", "step"):
        q = _exact_heads(s["new"][:, :nq], s.get("q_norm"), s["positions"])
        k = _exact_groups(_exact_heads(s["new"][:, nq:nq + h], s.get("k_norm"), s["positions"]), fmt, False)
        v = _exact_groups(s["new"][:, nq + h:].double(), fmt, True)
        if case["op"] == "write":
            return {"q": q, "k": k, "v": v}
        q = q.to(torch.bfloat16).double()[:, None]
    else:
        q = None if case["op"] == "read" else s["q"].double()
    outs, lses = [], []
    lens = _lengths(case)
    longest = max(1, s["max_len"])
    if case["op"] == "read":
        read_k, read_v = (torch.zeros(b, h, longest, d, dtype=torch.float64, device="cuda") for _ in range(2))
    begin = 0
    for i, n in enumerate(lens):
        ki = _exact_groups(s["old_k"][begin:begin + n].double(), fmt, False)
        vi = _exact_groups(s["old_v"][begin:begin + n].double(), fmt, True)
        begin += n
        if case["op"] == "read":
            read_k[i, :, :n], read_v[i, :, :n] = ki.transpose(0, 1), vi.transpose(0, 1)
            continue
        if case["op"] == "step":
            ki[n - 1], vi[n - 1] = k[i].to(torch.bfloat16).double() if fmt == "bf16" else k[i], v[i]
        for j in range(m):
            see = max(0, n - (m - 1 - j))
            out, lse = torch.zeros(nq, d, dtype=torch.float64, device="cuda"), torch.full((nq,), -math.inf, dtype=torch.float64, device="cuda")
            if see:
                scores = torch.matmul(q[i, j].view(h, nq // h, d), ki[:see].permute(1, 2, 0)) / math.sqrt(d)
                lse = torch.logsumexp(scores, -1).view(nq)
                out = torch.matmul(torch.softmax(scores, -1), vi[:see].transpose(0, 1)).reshape(nq, d)
            if case["join"]:
                pair = torch.stack([lse, s["base_lse"][i, j].double()])
                share = torch.softmax(pair, 0)[..., None]
                out, lse = share[0] * out + share[1] * s["base_out"][i, j].double(), torch.logsumexp(pair, 0)
            outs.append(out)
            lses.append(lse)
    if case["op"] == "read":
        return {"k": read_k, "v": read_v}
    return {"out": torch.stack(outs).view(b, m, nq, d), "lse": torch.stack(lses).view(b, m, nq)}
