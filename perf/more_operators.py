"""Long-lived agents' operators as measured workloads: attention of whole
prompts, a sliding window with a few first tokens that stay visible, caches
held in 4 bits, positions with several axes.  By a case's "op":

* prompt: attention of prompts' tokens (packed one after the other) over their
          own keys and values and those before them, causal, with a window and
          first tokens where the case has them, joined with attention over the
          pool where "join" is set.
* window: attention of each sequence's newest tokens over its pages, each
          seeing the newest `window` tokens and the first `sinks` ones.
* attend: attention over pages that hold keys and values in 4 bits.
* import: a cache that is already rotated (a card's, another agent's) written
          into 4-bit pages; returns keys and values as the pages hold them.
* write:  new tokens' queries, keys and values turned to positions of three
          axes (time, height, width) and written into pages.

With `own` false everything is elementary torch arithmetic in 32 bits on plain
tensors (64 bits for angles, and for codes, whose values lie next to a border);
with `own` true it is the library's calls.
"""
import math

import torch

own = False

THETA = 500000.0
GROUP = 32
EPS = 1e-5


# --- cases -------------------------------------------------------------------

def _prompt(name, heads, kv_heads, dim, seqs, q_min, q_max, past_min=0, past_max=0, window=0, sinks=0, join=False):
    c = dict(op="prompt", heads=heads, kv_heads=kv_heads, dim=dim, seqs=seqs, q_min=q_min, q_max=q_max, past_min=past_min,
             past_max=past_max, window=window, sinks=sinks, join=join)
    return dict(c, name=name) if name else c


def _paged(name, op, fmt, heads, kv_heads, dim, page, seqs, len_min, len_max, q_tokens=1, window=0, sinks=0, axes="", norm=False):
    c = dict(op=op, fmt=fmt, heads=heads, kv_heads=kv_heads, dim=dim, page=page, seqs=seqs, len_min=len_min,
             len_max=len_max, q_tokens=q_tokens, window=window, sinks=sinks, axes=axes, norm=norm)
    return dict(c, name=name) if name else c


def listed():
    return [
        # 15 agents each get a short message and see it beside the shared pool: latency
        _prompt("prompt-15-messages", 32, 8, 128, 15, 17, 17, join=True),
        # an agent's long private prompt on a layer that sees a window and four first tokens
        _prompt("prompt-8k-window", 32, 8, 128, 1, 8192, 8192, window=1024, sinks=4),
        # the same kind of prompt twice as long on a layer that sees everything
        _prompt("prompt-16k", 32, 8, 128, 1, 16384, 16384),
        # a turn of 509 tokens over a long history that was read back from the cache
        _prompt("prompt-turn-over-32k", 32, 8, 128, 1, 509, 509, past_min=32768, past_max=32768),
        # a ragged handful without grouped heads, some with a history
        _prompt("prompt-ragged-d64", 32, 32, 64, 7, 37, 1851, past_min=0, past_max=700, window=256, sinks=17),
        # one decode step of 15 agents with 4K behind them, of which a window counts: latency
        _paged("window-15agents-4k", "window", "bf16", 32, 8, 128, 16, 15, 4096, 4096, window=1024, sinks=4),
        # four agents that have run for long: a quarter of 128K is looked at, in 4 bits
        _paged("window-128k-4bit", "window", "k4v4", 32, 8, 128, 64, 4, 131072, 131072, window=32768, sinks=16),
        # attention over four 32K caches held in 4 bits
        _paged("attend-32k-4bit", "attend", "k4v4", 32, 8, 128, 64, 4, 32768, 32768),
        # many ragged sequences, one query head per KV head, some of them empty
        _paged("attend-ragged-4bit", "attend", "k4v4", 32, 32, 64, 32, 64, 0, 1851),
        # a received cache of 8192 tokens put into an agent's 4-bit pages
        _paged("import-8k-4bit", "import", "k4v4", 0, 8, 128, 64, 1, 8192, 8192),
        # 15 agents' newest tokens, positions with three axes: latency
        _paged("write-15-axes", "write", "k8v8", 32, 8, 128, 16, 15, 1, 1, axes="interleaved", norm=True),
        # a prompt with pictures
        _paged("write-8k-axes", "write", "k8v4", 32, 8, 128, 64, 1, 8192, 8192, axes="sections"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, evenly by its logarithm."""
    return min(hi, max(lo, int(lo * 2 ** rng.uniform(0, math.log2(hi / lo + 1)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "window", "attend", "import", "write"])
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 16, 32])
    group = rng.choice([1, 2, 3, 4, 5, 8]) if kv_heads <= 8 else 1
    heads = kv_heads * group
    window = rng.choice([0, _spread(rng, 1, 9000)])
    sinks = rng.choice([0, 1, 4, _spread(rng, 1, 300)]) if window else 0
    if op == "prompt":
        seqs = _spread(rng, 1, 40)
        q_max = _spread(rng, 1, 12000)
        past_max = rng.choice([0, _spread(rng, 1, 40000)])
        while seqs * heads * q_max * (q_max + past_max) * dim > 32 * 16384 * 16384 * 128 // 2:
            seqs, q_max, past_max = max(1, seqs // 2), max(1, q_max * 3 // 4), past_max * 3 // 4
        q_min, past_min = rng.choice([0, 1, q_max // 3, q_max]), rng.choice([0, past_max // 2, past_max])
        return _prompt(None, heads, kv_heads, dim, seqs, min(q_min, q_max), q_max, past_min, past_max, window, sinks,
                       rng.random() < 0.3)
    q_tokens = rng.choice([1, 1, 1, 2, 5, 8]) if op in ("window", "attend") else 1
    seqs = _spread(rng, 1, 90)
    most = {"import": 30000 * 8 * 128, "write": 8192 * 8 * 128}.get(op, 120000 * 8 * 128 // max(1, q_tokens * group // 8))
    len_max = _spread(rng, 1, max(2, min(131072, most // (seqs * kv_heads * dim))))
    len_min = min(rng.choice([0, 1, len_max // 3, len_max]), len_max)
    page = rng.choice([16, 32, 64, 128])
    if op == "window":
        window = window or _spread(rng, 1, 9000)
        return _paged(None, op, rng.choice(["bf16", "k8v8", "k8v4", "k4v4"]), heads, kv_heads, dim, page, seqs, len_min,
                      len_max, q_tokens, window, sinks)
    if op == "write":
        return _paged(None, op, rng.choice(["bf16", "k8v8", "k8v4"]), heads, kv_heads, dim, page, seqs, len_min, len_max,
                      axes=rng.choice(["sections", "interleaved"]), norm=rng.random() < 0.5)
    return _paged(None, op, "k4v4", heads if op == "attend" else 0, kv_heads, dim, page, seqs, len_min, len_max, q_tokens)


def _over(lo, hi, n, turn):
    """n whole numbers spread over [lo, hi]; the first is hi."""
    return [hi - int((hi - lo) * ((i * turn) % 1.0) + (0.5 if i else 0)) if hi > lo else hi for i in range(n)]


def _lengths(case):
    """Pages: tokens of each sequence.  Prompts: (new tokens, tokens behind them) of each."""
    if case["op"] != "prompt":
        return _over(case["len_min"], case["len_max"], case["seqs"], 0.6180339887498949)
    return list(zip(_over(case["q_min"], case["q_max"], case["seqs"], 0.6180339887498949),
                    _over(case["past_min"], case["past_max"], case["seqs"], 0.7548776662466927)))


def _pair_bytes(case):
    """Bytes that one cached token of one KV head takes, keys and values."""
    d, g = case["dim"], case["dim"] // GROUP
    return {"bf16": 4 * d, "k8v8": 2 * d + 4 * g, "k8v4": d + d // 2 + 6 * g, "k4v4": d + 8 * g}[case["fmt"]]


def _seen(pos, window, sinks):
    """How many tokens the token at `pos` sees."""
    if not window or window > pos:
        return pos + 1
    return window + min(sinks, pos + 1 - window)


def work(case):
    nq, h, d, w, s = (case[k] for k in ("heads", "kv_heads", "dim", "window", "sinks"))
    if case["op"] == "prompt":
        nbytes = flops = 0
        for n, past in _lengths(case):
            first = max(0, past - w + 1) if w else 0  # keys that any of the queries sees
            keys = past + n - first + min(s, first) if n else 0
            nbytes += n * nq * (4 * d + 4) + keys * h * 4 * d + (n * nq * (4 * d + 4) if case["join"] else 0)
            flops += 4 * nq * d * sum(_seen(past + i, w, s) for i in range(n))
        return {"bytes": nbytes, "flops": flops}
    lens, m, c = _lengths(case), case["q_tokens"], _pair_bytes(case)
    total = sum(lens)
    if case["op"] == "import":
        return {"bytes": total * h * (8 * d + c), "flops": total * h * d * 8}
    if case["op"] == "write":
        nbytes = total * (nq + 2 * h) * d * 2 + total * nq * d * 2 + total * h * (c + 4 * d) + total * 32
        return {"bytes": nbytes, "flops": total * (nq + 2 * h) * d * 10}
    read = sum(n if not w or n < w + m else min(n, w + m - 1 + min(s, n - w - m + 1)) for n in lens)
    products = sum(_seen(n - m + i, w, s) for n in lens for i in range(m) if n - m + i >= 0)
    return {"bytes": read * h * c + len(lens) * m * nq * (4 * d + 4), "flops": 4 * products * nq * d}


# --- inputs --------------------------------------------------------------------

_FORMATS = {"bf16": "KVP_PAGES_BF16", "k8v8": "KVP_PAGES_K8V8", "k8v4": "KVP_PAGES_K8V4", "k4v4": "KVP_PAGES_K4V4"}


def _keys(n, h, d, g, strong=20.0):
    """Keys with a few strong channels per head."""
    k = torch.randn(n, h, d, generator=g, device="cuda")
    at = torch.rand(h, d, generator=g, device="cuda").argsort(dim=1)[:, :4]
    return (k * torch.ones(h, d, device="cuda").scatter_(1, at, strong)).to(torch.bfloat16)


def _values(n, h, d, g):
    """Heavier tails than a Gaussian's (Student's t, 5 degrees)."""
    z = torch.randn(n, h, d, generator=g, device="cuda")
    w = torch.zeros(n, h, d, device="cuda")
    for _ in range(5):
        w += torch.randn(n, h, d, generator=g, device="cuda").square_()
    return z.mul_(0.5).div_(w.mul_(0.2).sqrt_()).to(torch.bfloat16)


def _base(s, shape, g):
    """Attention over the pool, as it leaves it."""
    s["base_out"] = 0.1 * torch.randn(shape, generator=g, device="cuda")
    s["base_lse"] = 5.0 + torch.rand(shape[:-1], generator=g, device="cuda") * 3


def _prompt_inputs(case, seed):
    """The fused projection's output of the new tokens; where there is a history, keys
    and values as one cache [heads][tokens][dim], which is how it is read back."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    nq, h, d = case["heads"], case["kv_heads"], case["dim"]
    lens = _lengths(case)
    n, t = sum(a for a, _ in lens), sum(a + b for a, b in lens)
    s = dict(n=n, t=t, max_q=max(a for a, _ in lens), max_k=max(a + b for a, b in lens))
    first = [0]
    for a, _ in lens:
        first.append(first[-1] + a)
    k_first = [0]
    for a, b in lens:
        k_first.append(k_first[-1] + a + b)
    as_int = dict(dtype=torch.int32, device="cuda")
    s["q_first"], s["k_first"] = torch.tensor(first, **as_int), torch.tensor(k_first[:-1], **as_int)
    s["k_lens"] = torch.tensor([a + b for a, b in lens], **as_int)
    q = torch.randn(n, nq, d, generator=g, device="cuda").to(torch.bfloat16)
    k, v = _keys(t, h, d, g, 4.0), _values(t, h, d, g)
    if t == n:
        x = torch.cat([q, k, v], dim=1)
        s["q"], s["k"], s["v"] = x[:, :nq], x[:, nq:nq + h], x[:, nq + h:]
    else:
        s["q"] = q
        s["k"], s["v"] = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (k, v))
    if case["join"]:
        _base(s, (n, nq, d), g)
    return s


def _paged_inputs(case, seed):
    """What a model and its scheduler have in hand for the page calls."""
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
    s = dict(lens=lens_t, table=table, max_pages=max_pages, n_pages=n_pages, max_len=max(lens),
             slots=table[seq, index // p].long() * p + index % p)
    total = sum(lens)
    if case["op"] == "write":
        s["new"] = torch.cat([torch.randn(total, nq, d, generator=g, device="cuda").to(torch.bfloat16),
                              _keys(total, h, d, g), _values(total, h, d, g)], dim=1)
        # text, then a picture of 31 columns, whose tokens share their time
        start = 4096 + int(torch.randint(0, 1000, (1,), generator=g, device="cuda"))
        shown = index >= 5
        at = torch.where(shown, index - 5, 0)
        s["positions"] = torch.stack([start + torch.where(shown, 5, index), start + torch.where(shown, 5 + at // 31, index),
                                      start + torch.where(shown, 5 + at % 31, index)])
        if case["norm"]:
            s["q_norm"] = (0.5 + torch.rand(d, generator=g, device="cuda")).to(torch.bfloat16)
            s["k_norm"] = (0.5 + torch.rand(d, generator=g, device="cuda")).to(torch.bfloat16)
        return s
    s["k"], s["v"] = _keys(total, h, d, g, 4.0 if case["fmt"] == "k4v4" else 20.0), _values(total, h, d, g)
    if case["op"] != "import":
        s["q"] = torch.randn(b, m, nq, d, generator=g, device="cuda").to(torch.bfloat16)
    return s


def _inv_freq(d):
    return [THETA ** (-2.0 * i / d) for i in range(d // 2)]


def _pair_axes(case):
    """The axis that each pair of dims turns by."""
    pairs = case["dim"] // 2
    return [p % 3 if case["axes"] == "interleaved" else p * 3 // pairs for p in range(pairs)]


def prepare(case, seed):
    nq, h, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "prompt":
        s = _prompt_inputs(case, seed)
        s.update(case=case, scale=1.0 / math.sqrt(d))
        if own:
            _prepare_own_prompt(s)
        return s
    s = _paged_inputs(case, seed)
    s.update(case=case, scale=1.0 / math.sqrt(d))
    if own:
        _prepare_own_pages(s)
    else:
        n = s["n_pages"] * case["page"]
        s["freq"] = torch.tensor(_inv_freq(d), dtype=torch.float32, device="cuda")
        s["axes_of"] = torch.tensor(_pair_axes(case), device="cuda")
        s["kc"], s["vc"] = (torch.zeros(n, h, d, dtype=torch.bfloat16 if case["fmt"] == "bf16" else torch.int8, device="cuda")
                            for _ in range(2))
        for name in ("ks", "kz", "vs", "vz"):
            s[name] = torch.zeros(n, h, d // GROUP, dtype=torch.float16, device="cuda")
        if case["op"] in ("window", "attend"):
            _store(s, s["slots"], s["k"].float(), s["v"].float())
    if case["op"] in ("window", "attend"):
        del s["k"], s["v"], s["slots"]
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
    kc, ks, *kz = _code4(k) if fmt == "k4v4" else _code8(k)
    vc, vs, *vz = _code8(v) if fmt == "k8v8" else _code4(v)
    s["kc"][slots], s["ks"][slots], s["vc"][slots], s["vs"][slots] = kc, ks, vc, vs
    if kz:
        s["kz"][slots] = kz[0]
    if vz:
        s["vz"][slots] = vz[0]
    return _value(kc, ks, *kz).to(torch.bfloat16), _value(vc, vs, *vz).to(torch.bfloat16)


def _load(s, tokens):
    """Tokens [seqs, n] of the sequences, in 32 bits, and whether they are there."""
    p, fmt = s["case"]["page"], s["case"]["fmt"]
    there = (tokens >= 0) & (tokens < s["lens"].long()[:, None])
    t = torch.where(there, tokens, 0)
    at = s["table"].long().gather(1, t // p) * p + t % p
    if fmt == "bf16":
        k, v = s["kc"][at].float(), s["vc"][at].float()
    else:
        k = _value(s["kc"][at], s["ks"][at], s["kz"][at] if fmt == "k4v4" else None)
        v = _value(s["vc"][at], s["vs"][at], None if fmt == "k8v8" else s["vz"][at])
    return k, torch.where(there[:, :, None, None], v, 0.0), there


def _softmax_values(x, v, eq):
    """Weighted values and the log of the sum of scores x (-Inf: not seen) over the last axis."""
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    w = torch.exp(x.sub_(top))
    total = w.sum(-1, keepdim=True)
    out = torch.einsum(eq, w.div_(torch.where(total > 0, total, 1.0)), v)
    return out, (top + torch.log(total))[..., 0]


def _joined(s, out, lse):
    if not s["case"].get("join"):
        return out, lse
    both = torch.maximum(lse, s["base_lse"])
    both = both + torch.log(torch.exp(lse - both) + torch.exp(s["base_lse"] - both))
    return (torch.exp(lse - both)[..., None] * out + torch.exp(s["base_lse"] - both)[..., None] * s["base_out"]), both


def _sees(t, pos, window, sinks):
    """Whether the token at `pos` sees token t."""
    seen = t <= pos
    return seen & ((t > pos - window) | (t < sinks)) if window else seen


def _plain_prompt(s):
    case = s["case"]
    nq, h, d, b = case["heads"], case["kv_heads"], case["dim"], case["seqs"]
    i, t = torch.arange(s["max_q"], device="cuda"), torch.arange(s["max_k"], device="cuda")
    q_first, k_first, k_lens = (s[x].long() for x in ("q_first", "k_first", "k_lens"))
    n = q_first[1:] - q_first[:-1]
    q = s["q"][(q_first[:-1, None] + i).clamp(max=s["n"] - 1)].float()       # [b, i, nq, d]
    at = (k_first[:, None] + t).clamp(max=s["t"] - 1)
    k, v = s["k"][at].float(), s["v"][at].float()                             # [b, t, h, d]
    v = torch.where((t < k_lens[:, None])[:, :, None, None], v, 0.0)
    x = torch.einsum("bihgd,bthd->bhgit", (q * s["scale"]).view(b, -1, h, nq // h, d), k)
    pos = (k_lens - n)[:, None] + i                                            # [b, i]
    x.masked_fill_(~_sees(t, pos[:, :, None], case["window"], case["sinks"])[:, None, None], -math.inf)
    out, lse = _softmax_values(x, v, "bhgit,bthd->bihgd")
    new = i < n[:, None]
    out, lse = out.reshape(b, -1, nq, d)[new], lse.permute(0, 3, 1, 2).reshape(b, -1, nq)[new]
    out, lse = _joined(s, out, lse)
    return {"out": out.to(torch.bfloat16), "lse": lse}


def _plain_attend(s):
    """Over the tokens that some query of a sequence may see: all, or the first ones and the window."""
    case = s["case"]
    nq, h, d, m, w = case["heads"], case["kv_heads"], case["dim"], case["q_tokens"], case["window"]
    b, lens, q = case["seqs"], s["lens"].long(), s["q"].float()
    every = torch.arange(max(1, s["max_len"]), device="cuda")
    if not w or w + m + case["sinks"] >= s["max_len"]:
        tokens = every.expand(b, -1)
    else:
        first = (lens - (w + m - 1)).clamp(min=case["sinks"])
        tokens = torch.cat([every[: case["sinks"]].expand(b, -1), first[:, None] + torch.arange(w + m - 1, device="cuda")], 1)
    k, v, there = _load(s, tokens)
    x = torch.einsum("bmhgd,bthd->bhmgt", (q * s["scale"]).view(b, m, h, nq // h, d), k)
    pos = lens[:, None] - m + torch.arange(m, device="cuda")
    seen = _sees(tokens[:, None, :], pos[:, :, None], w, case["sinks"]) & there[:, None, :]
    x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    out, lse = _softmax_values(x, v, "bhmgt,bthd->bmhgd")
    return {"out": out.reshape(b, m, nq, d).to(torch.bfloat16), "lse": lse.permute(0, 2, 1, 3).reshape(b, m, nq)}


def _normed(x, w):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _turned(x, cos, sin):
    half = x.shape[-1] // 2
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _plain_write(s):
    case = s["case"]
    nq, h = case["heads"], case["kv_heads"]
    x = s["new"].float()
    angle = s["positions"][s["axes_of"]].T.double() * s["freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q = _turned(_normed(x[:, :nq], s.get("q_norm")), cos, sin).to(torch.bfloat16)
    k = _turned(_normed(x[:, nq:nq + h], s.get("k_norm")), cos, sin)
    k, v = _store(s, s["slots"], k, x[:, nq + h:])
    return {"q": q, "k": k, "v": v}


def _plain_import(s):
    k, v = _store(s, s["slots"], s["k"].float(), s["v"].float())
    return {"k": k, "v": v}


# --- the library's calls ------------------------------------------------------------

def _stream():
    return torch.cuda.current_stream()


def _prepare_own_prompt(s):
    import agent_shared_compressed_gb300 as kv
    case = s["case"]
    nq, h, d = case["heads"], case["kv_heads"], case["dim"]
    shape = kv.PromptShape(case["seqs"], s["n"], s["t"], nq, h, d)
    s.update(kv=kv, shape=shape, ws=torch.empty(kv.kvprompt_workspace_bytes(shape), dtype=torch.uint8, device="cuda"),
             error=torch.zeros(1, dtype=torch.int32, device="cuda"),
             out=torch.empty(s["n"], nq, d, dtype=torch.bfloat16, device="cuda"),
             lse=torch.empty(s["n"], nq, dtype=torch.float32, device="cuda"))


def _own_prompt(s):
    kv, case = s["kv"], s["case"]
    kv.check(kv.kvprompt_attend(s["shape"], s["q"], s["k"], s["v"], s["q_first"], s["k_first"], s["k_lens"], s["scale"],
                                case["window"], case["sinks"], s.get("base_out"), s.get("base_lse"), s["out"], s["lse"],
                                s["error"], s["ws"], s["ws"].numel(), _stream()))
    return {"out": s["out"], "lse": s["lse"]}


def _prepare_own_pages(s):
    import ctypes

    import agent_shared_compressed_gb300 as kv
    case = s["case"]
    nq, h, d, p, b, m = (case[k] for k in ("heads", "kv_heads", "dim", "page", "seqs", "q_tokens"))
    cfg = kv.PagesConfig(1, h, d, p, s["n_pages"], getattr(kv, _FORMATS[case["fmt"]]))
    size = kv.kvpages_bytes(cfg)
    pages = torch.empty(size, dtype=torch.uint8, device="cuda")
    kv.check(kv.kvpages_init(cfg, pages, size, _stream()), "init")
    pairs = d // 2
    s.update(kv=kv, cfg=cfg, pages=pages, freq=(ctypes.c_float * pairs)(*_inv_freq(d)),
             axes_of=(ctypes.c_uint8 * pairs)(*_pair_axes(case)))
    n = s["slots"].numel()
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    if case["op"] in ("write", "import"):
        s["k_out"], s["v_out"] = (torch.empty(n, h, d, **bf16) for _ in range(2))
        s["q_out"] = torch.empty(n, nq, d, **bf16)
        return
    if n:
        kv.check(kv.kvpages_append(pages, cfg, 0, n, 0, None, s["k"], s["v"], s["slots"], None, None, None, 0.0, 0, None, None,
                                   None, None, _stream()), "append")
    s["ws"] = torch.empty(kv.kvpages_attend_workspace_bytes(cfg, b, m, nq), dtype=torch.uint8, device="cuda")
    s["out"] = torch.empty(b, m, nq, d, **bf16)
    s["lse"] = torch.empty(b, m, nq, dtype=torch.float32, device="cuda")


def _own_attend(s):
    kv, case = s["kv"], s["case"]
    rest = (s["table"], s["max_pages"], s["lens"], None, None, s["out"], s["lse"], s["ws"], s["ws"].numel(), _stream())
    counts = (s["pages"], s["cfg"], 0, case["seqs"], case["q_tokens"], case["heads"], s["q"], s["scale"])
    if case["op"] == "window":
        kv.check(kv.kvpages_attend_window(*counts, case["window"], case["sinks"], *rest))
    else:
        kv.check(kv.kvpages_attend(*counts, *rest))
    return {"out": s["out"], "lse": s["lse"]}


def _own_write(s):
    kv, case, x = s["kv"], s["case"], s["new"]
    nq, h, d = case["heads"], case["kv_heads"], case["dim"]
    kv.check(kv.kvpages_append_axes(s["pages"], s["cfg"], 0, x.shape[0], nq, x[:, :nq], x[:, nq:nq + h], x[:, nq + h:],
                                    s["slots"], s["positions"], 3, s["axes_of"], s.get("q_norm"), s.get("k_norm"), EPS, d,
                                    s["freq"], s["q_out"], s["k_out"], s["v_out"], _stream()))
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _own_import(s):
    kv = s["kv"]
    kv.check(kv.kvpages_append(s["pages"], s["cfg"], 0, s["k"].shape[0], 0, None, s["k"], s["v"], s["slots"], None, None, None,
                               0.0, 0, None, None, s["k_out"], s["v_out"], _stream()))
    return {"k": s["k_out"], "v": s["v_out"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"prompt": _own_prompt, "import": _own_import, "write": _own_write}.get(op, _own_attend)(state)
    return {"prompt": _plain_prompt, "import": _plain_import, "write": _plain_write}.get(op, _plain_attend)(state)


# --- the definition in 64 bits ---------------------------------------------------------

def _exact_groups(x, bits):
    """What the cache holds for x (64 bits, [..., dim]) at 8 or 4 bits (16: before the rounding)."""
    if bits == 16:
        return x
    blocks = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    if bits == 4:
        low = blocks.min(-1, keepdim=True).values
        step = ((blocks.max(-1, keepdim=True).values - low) / 15).to(torch.float16).double()
        zero = low.to(torch.float16).double()
        n = ((blocks - zero) / step).round().clamp(0, 15)
        kept = torch.where(step == 0, zero.expand_as(blocks), n * step + zero)
    else:
        step = (blocks.abs().max(-1, keepdim=True).values / 127).to(torch.float16).double()
        n = (blocks / step).round().clamp(-127, 127)
        kept = torch.where(step == 0, torch.zeros_like(blocks), n * step)
    return kept.reshape(x.shape)


_BITS = {"bf16": (16, 16), "k8v8": (8, 8), "k8v4": (8, 4), "k4v4": (4, 4)}


def _exact_heads(x, weight, turns):
    """Norm and rotation of [tokens, heads, dim] in 64 bits: pairs (i, i + dim/2) as complex numbers."""
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
    d = x.shape[-1]
    y = torch.complex(x[..., : d // 2].contiguous(), x[..., d // 2:].contiguous()) * turns[:, None]
    return torch.cat([y.real, y.imag], -1)


def _exact_rows(q, k, v, pos, case):
    """Attention of q [n, heads, dim] at positions pos over k, v [t, kv heads, dim], in 64 bits."""
    n, nq, d = q.shape
    h = k.shape[1]
    out = torch.zeros(n, nq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, nq), -math.inf, dtype=torch.float64, device="cuda")
    if k.shape[0] == 0:
        return out, lse
    t = torch.arange(k.shape[0], device="cuda")
    for i in range(0, n, 1024):
        at = pos[i:i + 1024]
        lo = max(0, int(at[0]) - case["window"] + 1) if case["window"] and case["sinks"] == 0 else 0
        hidden = at[:, None] < t[None, lo:]
        if case["window"]:
            hidden = hidden | ((at[:, None] - case["window"] >= t[None, lo:]) & (t[None, lo:] >= case["sinks"]))
        for j in range(nq):
            c = j // (nq // h)
            scores = (q[i:i + 1024, j].double() @ k[lo:, c].double().T / math.sqrt(d)).masked_fill(hidden, -math.inf)
            lse[i:i + 1024, j] = torch.logsumexp(scores, -1)
            out[i:i + 1024, j] = torch.softmax(scores, -1).nan_to_num(0.0) @ v[lo:, c].double()
    return out, lse


def exact(case, seed):
    nq, h, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "prompt":
        s = _prompt_inputs(case, seed)
        outs, lses, begin, k_begin = [], [], 0, 0
        for n, past in _lengths(case):
            o, l = _exact_rows(s["q"][begin:begin + n], s["k"][k_begin:k_begin + n + past], s["v"][k_begin:k_begin + n + past],
                               past + torch.arange(n, device="cuda"), case)
            begin, k_begin = begin + n, k_begin + n + past
            outs.append(o)
            lses.append(l)
        out, lse = torch.cat(outs), torch.cat(lses)
        if case["join"]:
            pair = torch.stack([lse, s["base_lse"].double()])
            share = torch.softmax(pair, 0)[..., None]
            out, lse = share[0] * out + share[1] * s["base_out"].double(), torch.logsumexp(pair, 0)
        return {"out": out, "lse": lse}
    s = _paged_inputs(case, seed)
    k_bits, v_bits = _BITS[case["fmt"]]
    if case["op"] == "write":
        freq = torch.tensor(_inv_freq(d), dtype=torch.float32).double().cuda()
        along = torch.stack([s["positions"][a] for a in _pair_axes(case)], 1)
        turns = torch.polar(torch.ones(along.shape, dtype=torch.float64, device="cuda"), along.double() * freq)
        return {"q": _exact_heads(s["new"][:, :nq], s.get("q_norm"), turns),
                "k": _exact_groups(_exact_heads(s["new"][:, nq:nq + h], s.get("k_norm"), turns), k_bits),
                "v": _exact_groups(s["new"][:, nq + h:].double(), v_bits)}
    if case["op"] == "import":
        return {"k": _exact_groups(s["k"].double(), k_bits), "v": _exact_groups(s["v"].double(), v_bits)}
    outs, lses, begin, m = [], [], 0, case["q_tokens"]
    for i, n in enumerate(_lengths(case)):
        first = max(0, n - m - case["window"] + 1) if case["window"] else 0  # the window's keys, and the first ones
        keep = torch.cat([torch.arange(min(case["sinks"], first), device="cuda"), torch.arange(first, n, device="cuda")])
        ki, vi = (_exact_groups(s[x][begin:begin + n][keep].double(), bits) for x, bits in (("k", k_bits), ("v", v_bits)))
        begin += n
        for j in range(m):
            at = n - m + j
            seen = (keep <= at) & ((keep > at - case["window"]) | (keep < case["sinks"]) if case["window"] else keep >= 0)
            o, l = (_exact_rows(s["q"][i, j:j + 1], ki[seen], vi[seen], torch.full((1,), 1 << 40, device="cuda"),
                                dict(window=0, sinks=0)))
            outs.append(o)
            lses.append(l)
    return {"out": torch.cat(outs).view(-1, m, nq, d), "lse": torch.cat(lses).view(-1, m, nq)}
