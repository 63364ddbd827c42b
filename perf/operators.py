"""The prompt path's operators, measured: attention of new tokens over a cache,
the packed cache write with rotary positions, reading a cache back, and the
rotary table.

Every case is a dict of plain values; ``prepare`` makes its inputs on the GPU
from a seed, ``run`` makes one pass over them: with ``own`` false in elementary
torch operations, with ``own`` true through the library.  ``work`` counts the
bytes and operations that a pass cannot do without, ``exact`` states the result
in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

QMAX = {"e4m3": 448.0, "i8": 127.0}
T16 = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(name, op, **kw):
    c = dict(name=name, op=op)
    c.update(kw)
    return c


def listed():
    return [
        # attention ----------------------------------------------------------
        # two short first messages on a small multi-query model: one launch's latency
        _case("attn-tiny-f16", "attention", batch=2, q_lo=7, q_hi=33, ctx_lo=0, ctx_hi=0, lens=1,
              qh=4, kvh=1, d=64, q="f16", kv="f16", page=0, scales="tensor"),
        # whole prompts packed behind one another, grouped heads: the compute-bound end
        _case("attn-prompts-bf16", "attention", batch=4, q_lo=333, q_hi=8192, ctx_lo=0, ctx_hi=0,
              lens=2, qh=32, kvh=8, d=128, q="bf16", kv="bf16", page=0, scales="tensor"),
        # a serving step's chunks over a paged 8-bit cache, ragged, some of one token
        _case("attn-chunks-e4m3-paged", "attention", batch=8, q_lo=1, q_hi=512, ctx_lo=1000,
              ctx_hi=8192, lens=3, qh=64, kvh=8, d=128, q="f16", kv="e4m3", page=64,
              scales="tensor"),
        # a follow-up question of a few tokens on a very long document: few rows, a long axis
        _case("attn-long-mqa-e4m3", "attention", batch=4, q_lo=16, q_hi=64, ctx_lo=100000,
              ctx_hi=131008, lens=4, qh=16, kvh=1, d=128, q="f16", kv="e4m3", page=0,
              scales="tensor"),
        # a mixed batch (single tokens beside chunks) over an INT8 cache with a scale per token
        _case("attn-mixed-i8-token", "attention", batch=32, q_lo=1, q_hi=256, ctx_lo=16,
              ctx_hi=16384, lens=5, qh=32, kvh=8, d=128, q="bf16", kv="i8", page=16,
              scales="token"),
        # packed cache write ---------------------------------------------------
        # one decode step's new tokens, rotated and quantised: latency
        _case("append-decode-e4m3", "append", batch=64, q_lo=1, q_hi=1, ctx_lo=16, ctx_hi=2048,
              lens=6, qh=64, kvh=8, d=128, q="f16", kv="e4m3", page=64, scales="tensor", rot=128,
              pairs="half"),
        # whole prompts into a 16-bit cache
        _case("append-prompts-bf16", "append", batch=4, q_lo=333, q_hi=8192, ctx_lo=0, ctx_hi=0,
              lens=7, qh=32, kvh=8, d=128, q="bf16", kv="bf16", page=0, scales="tensor", rot=128,
              pairs="interleaved"),
        # odd chunks, half of each head rotated, INT8 with a scale per token
        _case("append-chunks-i8-token", "append", batch=8, q_lo=1, q_hi=1001, ctx_lo=0,
              ctx_hi=8192, lens=8, qh=32, kvh=8, d=128, q="f16", kv="i8", page=16,
              scales="token", rot=64, pairs="half"),
        # reading a cache back -------------------------------------------------
        # a batch's whole paged FP8 cache as f16 rows (moved to another layout or machine)
        _case("read-batch-e4m3-paged", "read", batch=64, q_lo=16, q_hi=16384, ctx_lo=0, ctx_hi=0,
              lens=9, kvh=8, d=128, q="f16", kv="e4m3", page=64, scales="tensor"),
        # three short sequences of an INT8 cache with a scale per token
        _case("read-small-i8-token", "read", batch=3, q_lo=5, q_hi=333, ctx_lo=0, ctx_hi=77,
              lens=10, kvh=2, d=64, q="bf16", kv="i8", page=16, scales="token"),
        # rotary table ---------------------------------------------------------
        # a long-context table, frequencies scaled by parts
        _case("table-131072", "table", positions=131072, rot=128, theta=500000.0,
              scaling="by_parts", factor=8.0),
        # an ordinary context's table for a 64-wide rotation
        _case("table-4096", "table", positions=4096, rot=64, theta=10000.0, scaling="none",
              factor=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(4, 1), (16, 1), (8, 8), (32, 8), (64, 8), (6, 2), (10, 2), (12, 12)]
KV = [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3"), ("f16", "i8"),
      ("bf16", "i8")]


def draw(rng):
    op = rng.choice(["attention"] * 4 + ["append"] * 2 + ["read"] * 2 + ["table"])
    if op == "table":
        scaling = rng.choice(["none", "linear", "by_parts"])
        return dict(op=op, positions=_log_int(rng, 100, 131072), rot=16 * rng.randint(1, 8),
                    theta=rng.choice([10000.0, 500000.0, 1000000.0]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.uniform(1.5, 32.0))
    q, kv = rng.choice(KV)
    c = dict(op=op, batch=_log_int(rng, 1, 32), lens=rng.randrange(1 << 20), q=q, kv=kv,
             d=rng.choice([64, 128, 128]), page=rng.choice([0, 0, 1, 8, 16, 64, 256]),
             scales=rng.choice(["tensor", "head", "token"]) if kv in QMAX else "tensor")
    qh, c["kvh"] = rng.choice(HEADS)
    if op == "read":
        c["q_hi"] = _log_int(rng, 16, 16384)
        c["ctx_hi"] = rng.choice([0, _log_int(rng, 1, 500)])
    else:
        c["qh"] = qh
        c["q_hi"] = _log_int(rng, 1, 4096)
        c["ctx_hi"] = rng.choice([0, _log_int(rng, 1, 32768)])
    if op == "append":
        c["rot"] = rng.choice([0, 32, c["d"] // 2, c["d"], c["d"]])
        c["pairs"] = rng.choice(["half", "interleaved"])
    c["q_lo"] = rng.randint(1, max(1, c["q_hi"] // 2))
    c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
    # no dearer than the largest listed case
    top_f, top_b = 4.5e11, 2.5e8
    while True:
        w = work(c)
        if w["flops"] <= top_f and w["bytes"] <= top_b:
            return c
        if c["batch"] > 1:
            c["batch"] = max(1, c["batch"] // 2)
        else:
            c["q_hi"] = max(1, c["q_hi"] // 2)
            c["q_lo"] = min(c["q_lo"], c["q_hi"])


def _lengths(c):
    """(new or read tokens, context before them) per sequence: the case's own,
    log-uniform between its bounds, which both occur."""
    r = np.random.RandomState(c["lens"])

    def some(lo, hi):
        v = np.exp(r.uniform(math.log(lo + 1), math.log(hi + 2), c["batch"])).astype(np.int64) - 1
        v = np.clip(v, lo, hi)
        v[-1], v[0] = lo, hi
        return [int(x) for x in v]

    return some(c["q_lo"], c["q_hi"]), some(c["ctx_lo"], c["ctx_hi"])[::-1]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _starts(lens):
    return [0] + [int(x) for x in np.cumsum(lens)]


def _placement(c, seq, gen, dev):
    """Where the sequences' rows lie: block table (a random permutation of a
    1.2 times oversized pool) or first rows (a gap of three rows between
    sequences), and the number of cache rows."""
    if c["page"]:
        P = c["page"]
        need = [-(-t // P) for t in seq]
        pool = max(1, int(math.ceil(1.2 * sum(need))))
        perm = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
        stride = max(1, max(need))
        at = torch.tensor(_starts(need)[:-1], device=dev)[:, None] + torch.arange(stride, device=dev)
        table = perm[at.clamp_(max=pool - 1)].contiguous()
        return table, None, pool * P
    starts = _starts([t + 3 for t in seq])
    return None, torch.tensor(starts[:-1], dtype=torch.int32, device=dev), starts[-1]


def _normal(shape, dtype, gen, dev):
    return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)


def _cache_shape(c, rows):
    return (rows // c["page"], c["page"], c["kvh"], c["d"]) if c["page"] else (rows, c["kvh"], c["d"])


def _filled(c, rows, gen, dev):
    """A cache holding N(0, 1) values in the case's format: (codes, scale per
    tensor, finer scales)."""
    x = torch.randn((rows, c["kvh"], c["d"]), generator=gen, device=dev)
    if c["kv"] not in QMAX:
        return x.to(T16[c["kv"]]).view(_cache_shape(c, rows)), 1.0, None
    qmax = QMAX[c["kv"]]
    scale = 5.0 / qmax
    fine = None
    if c["scales"] == "head":
        fine = torch.rand(c["kvh"], generator=gen, device=dev) + 0.5
        x = x / (scale * fine[None, :, None])
    elif c["scales"] == "token":
        fine = torch.rand((rows, c["kvh"]), generator=gen, device=dev) + 0.5
        x = x / (scale * fine[:, :, None])
    else:
        x = x / scale
    x = x.clamp_(-qmax, qmax)
    codes = x.to(torch.float8_e4m3fn).view(torch.uint8) if c["kv"] == "e4m3" else \
        x.round_().to(torch.int8)
    return codes.view(_cache_shape(c, rows)), scale, fine


def _table64(c, dev):
    """cos and sin of every position, in 64 bits: [positions, rot]."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device=dev)
    f = c["theta"] ** (-2.0 * i / c["rot"])
    if c["scaling"] == "linear":
        f = f / c["factor"]
    elif c["scaling"] == "by_parts":
        turns = 8192.0 * f / (2.0 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        f = (1.0 - keep) * f / c["factor"] + keep * f
    a = torch.arange(c["positions"], dtype=torch.float64, device=dev)[:, None] * f
    return torch.cat([a.cos(), a.sin()], dim=1)


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    if c["op"] == "table":
        # the inputs are the settings; the seed moves theta a little
        theta = c["theta"] * (1.0 + (seed % 997) * 1e-4)
        return dict(case=c, op=c["op"], settings=dict(c, theta=theta))
    new, ctx = _lengths(c)
    seq = [a + b for a, b in zip(new, ctx)]
    table, first_row, rows = _placement(c, seq, gen, dev)
    i32 = dict(dtype=torch.int32, device=dev)
    s = dict(case=c, op=c["op"], new=new, ctx=ctx, rows=rows, block_table=table,
             kv_start_idx=first_row, q_start=torch.tensor(_starts(new), **i32),
             seq_len=torch.tensor(seq, **i32), positions=torch.tensor(ctx, **i32))
    total, t16 = sum(new), T16[c["q"]]
    if c["op"] == "append":
        s["q"] = _normal((total, c["qh"], c["d"]), t16, gen, dev)
        s["k_new"] = _normal((total, c["kvh"], c["d"]), t16, gen, dev)
        s["v_new"] = _normal((total, c["kvh"], c["d"]), t16, gen, dev)
        store = T16.get(c["kv"]) or (torch.uint8 if c["kv"] == "e4m3" else torch.int8)
        s["k"] = torch.zeros(_cache_shape(c, rows), dtype=store, device=dev)
        s["v"] = torch.zeros(_cache_shape(c, rows), dtype=store, device=dev)
        s["k_scale"] = s["v_scale"] = 5.0 / QMAX[c["kv"]] if c["kv"] in QMAX else 1.0
        s["k_scales"] = s["v_scales"] = None
        if c["scales"] == "head":
            s["k_scales"] = torch.rand(c["kvh"], generator=gen, device=dev) + 0.5
            s["v_scales"] = torch.rand(c["kvh"], generator=gen, device=dev) + 0.5
        elif c["scales"] == "token":
            s["k_scales"] = torch.ones((rows, c["kvh"]), device=dev)
            s["v_scales"] = torch.ones((rows, c["kvh"]), device=dev)
        s["rotary"] = None
        if c["rot"]:
            s["rotary"] = _table64(dict(rot=c["rot"], theta=10000.0, scaling="none",
                                        positions=max(seq)), dev).float()
        return s
    if c["op"] == "attention":
        s["q"] = _normal((total, c["qh"], c["d"]), t16, gen, dev)
    s["k"], s["k_scale"], s["k_scales"] = _filled(c, rows, gen, dev)
    s["v"], s["v_scale"], s["v_scales"] = _filled(c, rows, gen, dev)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _rows_of(s, b, lo, hi):
    """Cache rows of tokens lo .. hi - 1 of sequence b."""
    t = torch.arange(lo, hi, device="cuda")
    if s["block_table"] is None:
        return s["kv_start_idx"][b].long() + t
    P = s["case"]["page"]
    return s["block_table"][b].long()[t // P] * P + t % P


def _new_rows(s):
    """Cache rows of every packed token, and their positions."""
    seq = torch.repeat_interleave(torch.arange(len(s["new"]), device="cuda"),
                                  s["q_start"][1:] - s["q_start"][:-1], output_size=sum(s["new"]))
    pos = s["positions"][seq] + torch.arange(len(seq), device="cuda") - s["q_start"][seq]
    if s["block_table"] is None:
        return s["kv_start_idx"][seq].long() + pos, pos
    P = s["case"]["page"]
    return s["block_table"][seq, pos // P].long() * P + pos % P, pos


def _values(s, which, rows, dtype):
    """The values of cache rows, in `dtype`: [rows, KVH, D]."""
    c = s["case"]
    x = s[which].view(-1, c["kvh"], c["d"])[rows]
    if c["kv"] == "e4m3":
        x = x.view(torch.float8_e4m3fn)
    x = x.to(dtype)
    if c["kv"] in QMAX:
        scale, fine = s[which + "_scale"], s[which + "_scales"]
        if c["scales"] == "head":
            x = x * (scale * fine)[None, :, None]
        elif c["scales"] == "token":
            x = x * (scale * fine[rows])[:, :, None]
        else:
            x = x * scale
    return x


def _plain_attention(s):
    c = s["case"]
    out, lse, at = torch.empty_like(s["q"]), [], 0
    G = c["qh"] // c["kvh"]
    for b, (n, ctx) in enumerate(zip(s["new"], s["ctx"])):
        rows = _rows_of(s, b, 0, n + ctx)
        k, v = (_values(s, w, rows, torch.float32).transpose(0, 1) for w in "kv")
        q = s["q"][at:at + n].float().view(n, c["kvh"], G, c["d"])
        q = q.permute(1, 2, 0, 3).reshape(c["kvh"], G * n, c["d"])
        score = (torch.bmm(q, k.transpose(1, 2)) * c["d"] ** -0.5).view(c["kvh"], G, n, n + ctx)
        late = torch.arange(n + ctx, device="cuda") > ctx + torch.arange(n, device="cuda")[:, None]
        score.masked_fill_(late, -math.inf)
        m = score.amax(-1, keepdim=True)
        score.sub_(m).exp_()
        z = score.sum(-1, keepdim=True)
        o = torch.bmm(score.view(c["kvh"], G * n, n + ctx), v).view(c["kvh"], G, n, c["d"]) / z
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, c["qh"], c["d"])
        lse.append((m + z.log()).squeeze(-1).permute(2, 0, 1).reshape(n, c["qh"]))
        at += n
    return {"out": out, "lse": torch.cat(lse)}


def _rotate(x, table, pos, rot, pairs):
    """x: [tokens, heads, D] in 32 bits; the first `rot` dims of every head turned."""
    cs = table[pos][:, None, :]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    y = x.clone()
    if pairs == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    return y


def _f32(x):
    return torch.full((), x, dtype=torch.float32, device="cuda")


def _plain_append(s):
    c = s["case"]
    rows, pos = _new_rows(s)
    q, k = s["q"], s["k_new"].float()
    if c["rot"]:
        q = _rotate(q.float(), s["rotary"], pos, c["rot"], c["pairs"]).to(q.dtype)
        k = _rotate(k, s["rotary"], pos, c["rot"], c["pairs"])
    res = {"q": q}
    for w, x in (("k", k), ("v", s["v_new"].float())):
        cache = s[w].view(-1, c["kvh"], c["d"])
        if c["kv"] not in QMAX:
            cache[rows] = x.to(cache.dtype)
            res[w] = s[w]
            continue
        qmax, scale = QMAX[c["kv"]], _f32(s[w + "_scale"])
        if c["scales"] == "head":
            by = (scale * s[w + "_scales"])[None, :, None]
        elif c["scales"] == "token":
            amax = x.abs().amax(-1)
            fine = torch.where(amax > 0, amax / (qmax * scale), 1.0)
            s[w + "_scales"][rows] = fine
            by = (scale * fine)[:, :, None]
            res[w + "_scales"] = s[w + "_scales"]
        else:
            by = scale
        x = (x / by).clamp(-qmax, qmax)
        if c["kv"] == "e4m3":
            cache[rows] = x.to(torch.float8_e4m3fn).view(torch.uint8)
            res[w] = s[w].view(torch.float8_e4m3fn)
        else:
            cache[rows] = x.round().to(torch.int8)
            res[w] = s[w]
    return res


def _plain_read(s):
    rows, _ = _new_rows(s)
    t16 = T16[s["case"]["q"]]
    return {w: _values(s, w, rows, torch.float32).to(t16) for w in "kv"}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _own(s):
    import flash_decoding_attention_gb300 as fda
    c = s["case"]
    if s["op"] == "table":
        t = s["settings"]
        return {"table": fda.rotary_table(t["positions"], t["rot"], theta=t["theta"],
                                          scaling=t["scaling"], factor=t["factor"],
                                          original_positions=8192, low_turns=1.0, high_turns=4.0)}
    if "workspace" not in s:   # a serving program keeps it from step to step
        s["workspace"] = fda.alloc_prefill_workspace(c["d"])
    kw = dict(kv_start_idx=s["kv_start_idx"], block_table=s["block_table"], k_scale=s["k_scale"],
              v_scale=s["v_scale"], k_scales=s["k_scales"], v_scales=s["v_scales"],
              workspace=s["workspace"])
    if s["op"] == "attention":
        out, lse = fda.prefill_attention(s["q"], s["k"], s["v"], s["q_start"], s["seq_len"], **kw)
        return {"out": out, "lse": lse}
    if s["op"] == "read":
        k, v = fda.read_kv(s["k"], s["v"], s["q_start"], sum(s["new"]), first=s["positions"],
                           dtype=T16[c["q"]], **kw)
        return {"k": k, "v": v}
    q = fda.append_kv(s["k_new"], s["v_new"], s["k"], s["v"], s["q_start"], s["positions"],
                      q=s["q"], rotary=s["rotary"], interleaved=c["pairs"] == "interleaved", **kw)
    res = {"q": q, "k": s["k"], "v": s["v"]}
    if c["kv"] == "e4m3":
        res["k"], res["v"] = s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn)
    if c["scales"] == "token":
        res["k_scales"], res["v_scales"] = s["k_scales"], s["v_scales"]
    return res


def run(state):
    s = state
    if own:
        return _own(s)
    if s["op"] == "table":
        return {"table": _table64(s["settings"], "cuda").float()}
    if s["op"] == "attention":
        return _plain_attention(s)
    return _plain_append(s) if s["op"] == "append" else _plain_read(s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "table":
        return {"bytes": 4 * c["positions"] * c["rot"], "flops": 2 * c["positions"] * c["rot"]}
    new, ctx = _lengths(c)
    total = sum(new)
    code = 1 if c["kv"] in QMAX else 2
    per_row = 2 * c["kvh"] * (c["d"] * code + (4 if c["scales"] == "token" else 0))
    if c["op"] == "read":
        return {"bytes": total * (per_row + 2 * c["kvh"] * c["d"] * 2),
                "flops": 2 * total * c["kvh"] * c["d"]}
    if c["op"] == "append":
        rows = total * 2 * (c["qh"] + 2 * c["kvh"]) * c["d"]
        back = total * (2 * c["qh"] * c["d"] + per_row)
        turned = 4 * c["rot"] * len({p for n, x in zip(new, ctx) for p in range(x, x + n)})
        return {"bytes": rows + back + turned,
                "flops": total * (3 * (c["qh"] + c["kvh"]) * c["rot"] + 2 * c["kvh"] * c["d"])}
    seen = sum(n * x + n * (n + 1) // 2 for n, x in zip(new, ctx))
    kv = sum(n + x for n, x in zip(new, ctx)) * per_row
    return {"bytes": kv + total * c["qh"] * (4 * c["d"] + 4), "flops": 4 * seen * c["qh"] * c["d"]}


# ---------------------------------------------------------------------------
# the same results from their definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_rows(s, b):
    """Cache row of every token of sequence b, counted out on the host."""
    n = s["new"][b] + s["ctx"][b]
    if s["block_table"] is None:
        first = int(s["kv_start_idx"][b])
        return [first + t for t in range(n)]
    P, pages = s["case"]["page"], s["block_table"][b].tolist()
    return [pages[t // P] * P + t % P for t in range(n)]


def _exact_values(s, which, at):
    c = s["case"]
    codes = s[which].reshape(-1, c["kvh"], c["d"])[at]
    x = (codes.view(torch.float8_e4m3fn) if c["kv"] == "e4m3" else codes).double()
    if c["kv"] in QMAX:
        x = x * float(np.float32(s[which + "_scale"]))
        if s[which + "_scales"] is not None:
            f = s[which + "_scales"].double()
            x = x * (f if c["scales"] == "head" else f[at])[..., None]
    return x


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "table":
        t = s["settings"]
        dims = np.arange(t["rot"] // 2, dtype=np.float64)
        f = np.exp(-2.0 * dims / t["rot"] * math.log(t["theta"]))
        if t["scaling"] == "by_parts":
            ramp = np.clip((8192.0 * f / (2.0 * np.pi) - 1.0) / 3.0, 0.0, 1.0)
            f = f * (ramp + (1.0 - ramp) / t["factor"])
        elif t["scaling"] == "linear":
            f = f / t["factor"]
        angle = np.outer(np.arange(t["positions"], dtype=np.float64), f)
        return {"table": np.concatenate([np.cos(angle), np.sin(angle)], axis=1)}
    if c["op"] == "attention":
        G, outs, lses, at = c["qh"] // c["kvh"], [], [], 0
        for b, (n, ctx) in enumerate(zip(s["new"], s["ctx"])):
            rows = torch.tensor(_exact_rows(s, b), device="cuda")
            k, v = _exact_values(s, "k", rows), _exact_values(s, "v", rows)
            q = s["q"][at:at + n].double()
            o = torch.empty_like(q)
            l = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
            keys = torch.arange(n + ctx, device="cuda")
            for lo in range(0, n, 2048):   # some queries at a time
                hi = min(n, lo + 2048)
                hidden = keys[None, :] > (ctx + torch.arange(lo, hi, device="cuda"))[:, None]
                for h in range(c["qh"]):
                    e = q[lo:hi, h] @ k[:, h // G].T / math.sqrt(c["d"])
                    e[hidden] = -math.inf
                    l[lo:hi, h] = torch.logsumexp(e, 1)
                    o[lo:hi, h] = torch.exp(e - l[lo:hi, h, None]) @ v[:, h // G]
            outs.append(o)
            lses.append(l)
            at += n
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    rows, pos = [], []
    for b, (n, ctx) in enumerate(zip(s["new"], s["ctx"])):
        rows += _exact_rows(s, b)[ctx:]
        pos += range(ctx, ctx + n)
    rows = torch.tensor(rows, device="cuda")
    if c["op"] == "read":
        return {w: _exact_values(s, w, rows) for w in "kv"}
    q, k, v = s["q"].double(), s["k_new"].double(), s["v_new"].double()
    if c["rot"]:
        half = c["rot"] // 2
        t = s["rotary"].double()[torch.tensor(pos, device="cuda")]
        turn = torch.complex(t[:, :half], t[:, half:])[:, None, :]
        for x in (q, k):
            if c["pairs"] == "half":
                z = torch.complex(x[..., :half], x[..., half:c["rot"]].contiguous()) * turn
                x[..., :half], x[..., half:c["rot"]] = z.real, z.imag
            else:
                z = torch.complex(x[..., 0:c["rot"]:2], x[..., 1:c["rot"]:2]) * turn
                x[..., 0:c["rot"]:2], x[..., 1:c["rot"]:2] = z.real, z.imag
    res = {"q": q}
    for w, x in (("k", k), ("v", v)):
        full = torch.zeros(s[w].shape, dtype=torch.float64, device="cuda")
        if c["kv"] in QMAX:
            step = torch.full(x.shape[:2], float(np.float32(s[w + "_scale"])), dtype=torch.float64,
                              device="cuda")
            if c["scales"] == "head":
                step = step * s[w + "_scales"].double()
            elif c["scales"] == "token":
                fine = x.abs().amax(-1) / (QMAX[c["kv"]] * step)
                fine[fine == 0] = 1.0
                step = step * fine
                res[w + "_scales"] = torch.ones(s[w + "_scales"].shape, dtype=torch.float64,
                                                device="cuda")
                res[w + "_scales"][rows] = fine
            x = (x / step[..., None]).clamp(-QMAX[c["kv"]], QMAX[c["kv"]])
        full.view(-1, c["kvh"], c["d"])[rows] = x
        # INT8 codes are whole numbers: no value between them is an answer
        res[w] = None if c["kv"] == "i8" else full
    return res
