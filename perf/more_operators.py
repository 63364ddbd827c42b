"""A sliding-window serving step's operators, measured: attention that sees a
window and a few first tokens (single tokens, and packed prompts and chunks),
the packed cache write with per-head norms and rotary positions on several
axes, and the block tables and slot maps of a step's requests.

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
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(name, op, **kw):
    c = dict(name=name, op=op)
    c.update(kw)
    return c


def listed():
    return [
        # one token per sequence -----------------------------------------------
        # a small grouped model's first answers, windows barely filled: latency
        _case("decode-small-bf16", "decode", batch=4, ctx_lo=1, ctx_hi=700, lens=1, qh=8, kvh=2,
              d=64, q="bf16", kv="bf16", page=0, scales="tensor", window=512, sinks=4),
        # a full serving batch over a paged 8-bit cache, long and short sequences
        _case("decode-batch-e4m3-paged", "decode", batch=64, ctx_lo=256, ctx_hi=32768, lens=2,
              qh=64, kvh=8, d=128, q="f16", kv="e4m3", page=64, scales="tensor", window=4096,
              sinks=4),
        # few very long documents, one KV head, an INT8 cache with a scale per token
        _case("decode-long-mqa-i8-token", "decode", batch=16, ctx_lo=100000, ctx_hi=131008, lens=3,
              qh=16, kvh=1, d=128, q="bf16", kv="i8", page=0, scales="token", window=8191,
              sinks=64),
        # packed prompts and chunks --------------------------------------------
        # two short first messages, a window shorter than the longer one: latency
        _case("prefill-small-f16", "prefill", batch=2, q_lo=7, q_hi=333, ctx_lo=0, ctx_hi=0, lens=4,
              qh=4, kvh=1, d=64, q="f16", kv="f16", page=0, scales="tensor", window=65, sinks=1),
        # whole prompts of a local layer
        _case("prefill-prompts-bf16", "prefill", batch=4, q_lo=333, q_hi=8192, ctx_lo=0, ctx_hi=0,
              lens=5, qh=32, kvh=8, d=128, q="bf16", kv="bf16", page=0, scales="tensor",
              window=1024, sinks=0),
        # a step's chunks, some of one token, over long contexts in a paged 8-bit cache
        _case("prefill-chunks-e4m3-paged", "prefill", batch=8, q_lo=1, q_hi=2048, ctx_lo=1000,
              ctx_hi=32768, lens=6, qh=64, kvh=8, d=128, q="f16", kv="e4m3", page=16,
              scales="tensor", window=4096, sinks=16),
        # packed cache write with norms and axes -------------------------------
        # one decode step's new tokens, normed, rotated and quantised: latency
        _case("append-decode-norm-e4m3", "append", batch=64, q_lo=1, q_hi=1, ctx_lo=16, ctx_hi=2048,
              lens=7, qh=64, kvh=8, d=128, q="f16", kv="e4m3", page=64, scales="tensor", rot=128,
              pairs="half", norm="q", axes="none"),
        # whole text prompts into a 16-bit cache, norm weights kept in 32 bits
        _case("append-prompts-norm-bf16", "append", batch=4, q_lo=333, q_hi=8192, ctx_lo=0,
              ctx_hi=0, lens=8, qh=32, kvh=8, d=128, q="bf16", kv="bf16", page=0, scales="tensor",
              rot=128, pairs="half", norm="f32", axes="none"),
        # images between text, time, height and width in runs of pairs, INT8 with a scale per token
        _case("append-images-axes-i8", "append", batch=8, q_lo=1, q_hi=1001, ctx_lo=0, ctx_hi=8192,
              lens=9, qh=32, kvh=8, d=128, q="f16", kv="i8", page=16, scales="token", rot=128,
              pairs="half", norm="q", axes="runs"),
        # a video's frames, axes taking turns over neighbouring pairs, half of each head, no norm
        _case("append-video-axes-bf16", "append", batch=2, q_lo=4000, q_hi=6000, ctx_lo=0,
              ctx_hi=100, lens=10, qh=16, kvh=4, d=128, q="bf16", kv="bf16", page=256,
              scales="tensor", rot=64, pairs="interleaved", norm="none", axes="turns"),
        # block tables and slot maps -------------------------------------------
        # a decode step: one token each, now and then a page, pages behind the window go back
        _case("pages-decode-step", "pages", batch=256, new_lo=1, new_hi=1, ctx_lo=16, ctx_hi=8192,
              lens=11, page=16, window=1024, sinks=4, ended=0.02, short=False),
        # many requests admitted at once beside ended ones, with too few pages for all
        _case("pages-admit-prompts", "pages", batch=1024, new_lo=1, new_hi=8192, ctx_lo=0,
              ctx_hi=4096, lens=12, page=16, window=0, sinks=0, ended=0.25, short=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(4, 1), (16, 1), (8, 8), (32, 8), (64, 8), (6, 2), (10, 2), (12, 12)]
KV = [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3"), ("f16", "i8"),
      ("bf16", "i8")]


def draw(rng):
    op = rng.choice(["decode"] * 3 + ["prefill"] * 3 + ["append"] * 3 + ["pages"] * 2)
    if op == "pages":
        hi = rng.choice([1, 1, _log_int(rng, 2, 8192)])
        return dict(op=op, batch=_log_int(rng, 1, 1024), new_lo=rng.randint(min(1, hi - 1), 1),
                    new_hi=hi, ctx_lo=0, ctx_hi=_log_int(rng, 1, 4096), lens=rng.randrange(1 << 20),
                    page=rng.choice([1, 8, 16, 64, 256]) if hi < 100 else rng.choice([16, 64, 256]),
                    window=rng.choice([0, _log_int(rng, 1, 2048)]), sinks=rng.choice([0, 4, 33]),
                    ended=rng.choice([0.0, 0.1, 0.5]), short=rng.random() < 0.5)
    q, kv = rng.choice(KV)
    c = dict(op=op, batch=_log_int(rng, 1, 64), lens=rng.randrange(1 << 20), q=q, kv=kv,
             d=rng.choice([64, 128, 128]), page=rng.choice([0, 0, 1, 8, 16, 64, 256]),
             scales=rng.choice(["tensor", "head", "token"]) if kv in QMAX else "tensor")
    qh, kvh = rng.choice(HEADS)
    c["qh"], c["kvh"] = qh, kvh
    if op == "decode":
        c["ctx_hi"] = _log_int(rng, 1, 131072)
    else:
        c["batch"] = min(c["batch"], 32)
        c["q_hi"] = _log_int(rng, 1, 4096)
        c["q_lo"] = rng.randint(1, max(1, c["q_hi"] // 2))
        c["ctx_hi"] = rng.choice([0, _log_int(rng, 1, 32768)])
    c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
    if op == "append":
        c["rot"] = rng.choice([0, 32, c["d"] // 2, c["d"], c["d"]])
        c["pairs"] = rng.choice(["half", "interleaved"])
        c["norm"] = rng.choice(["none", "q", "f32", "f32"])
        c["axes"] = rng.choice(["none", "runs", "turns"]) if c["rot"] else "none"
    else:
        c["window"] = _log_int(rng, 1, 8192)
        c["sinks"] = rng.choice([0, 0, 1, 4, _log_int(rng, 1, 300)])
    # no dearer than the largest listed one
    top_f, top_b, top_rows = 2.4e11, 2.5e8, 2.0e6
    while True:
        w = work(c)
        new, ctx = _lengths(c)
        if w["flops"] <= top_f and w["bytes"] <= top_b and sum(new) + sum(ctx) <= top_rows / c["kvh"] ** 0.5:
            return c
        if c["batch"] > 1:
            c["batch"] = max(1, c["batch"] // 2)
        elif op == "decode":
            c["ctx_hi"] = max(1, c["ctx_hi"] // 2)
        else:
            c["q_hi"] = max(1, c["q_hi"] // 2)
            c["q_lo"] = min(c["q_lo"], c["q_hi"])
        c["ctx_lo"] = min(c["ctx_lo"], c["ctx_hi"])


def _lengths(c):
    """(new tokens, context before them) per sequence: the case's own,
    log-uniform between its bounds, which both occur."""
    r = np.random.RandomState(c["lens"])

    def some(lo, hi):
        v = np.exp(r.uniform(math.log(lo + 1), math.log(hi + 2), c["batch"])).astype(np.int64) - 1
        v = np.clip(v, lo, hi)
        v[-1], v[0] = lo, hi
        return [int(x) for x in v]

    lo, hi = (1, 1) if c["op"] == "decode" else \
        (c["new_lo"], c["new_hi"]) if c["op"] == "pages" else (c["q_lo"], c["q_hi"])
    new, ctx = some(lo, hi), some(c["ctx_lo"], c["ctx_hi"])[::-1]
    if c["op"] == "decode":   # the context counts the new token
        ctx = [max(0, x - 1) for x in ctx]
    if c["op"] == "pages":
        gone = r.uniform(size=c["batch"]) < c["ended"]
        new = [-1 if g else n for g, n in zip(gone, new)]
    return new, ctx


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
        return perm[at.clamp_(max=pool - 1)].contiguous(), None, pool * P
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


def _table64(rot, positions, dev):
    """cos and sin of every position, in 64 bits: [positions, rot]."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=dev)
    a = torch.arange(positions, dtype=torch.float64, device=dev)[:, None] * 10000.0 ** (-2.0 * i / rot)
    return torch.cat([a.cos(), a.sin()], dim=1)


def _pair_axes(c):
    """Axis of every rotary pair: a quarter, three eighths and three eighths in
    runs, or taking turns."""
    n = c["rot"] // 2
    if c["axes"] == "turns":
        return [i % 3 for i in range(n)]
    return [0 if i < n // 4 else 1 if i < n // 4 + 3 * n // 8 else 2 for i in range(n)]


def _axis_positions(total, seed, dev):
    """Time, height and width of every token: stretches of text, whose three
    positions go on together, between images of up to 32 x 32 patches."""
    r = np.random.RandomState(seed % (1 << 31))
    parts, have, at = [], 0, int(r.randint(0, 50))
    while have < total:
        if r.uniform() < 0.4:
            n = int(r.randint(1, 200))
            p = np.broadcast_to(at + np.arange(n), (3, n))
            at += n
        else:
            h, w = int(r.randint(2, 33)), int(r.randint(2, 33))
            p = at + np.stack([np.zeros(h * w, np.int64), np.repeat(np.arange(h), w),
                               np.tile(np.arange(w), h)])
            at += max(h, w)
        parts.append(p)
        have += p.shape[1]
    p = np.ascontiguousarray(np.concatenate(parts, 1)[:, :total]).astype(np.int32)
    return torch.from_numpy(p).to(dev), int(p.max()) + 1


def _gone(c, x):
    """First column that is not given back yet when x tokens are cached, as the
    step before left it."""
    return max(-(-c["sinks"] // c["page"]), max(0, x - c["window"]) // c["page"])


def _prepare_pages(c, seed, gen, dev):
    """A server's page state: block tables of the running requests, the stack
    of free pages, and this step's new tokens per request (-1: it has ended)."""
    new, ctx = _lengths(c)
    if seed % 2:   # another seed, another order of the requests
        new, ctx = new[::-1], ctx[::-1]
    P = c["page"]
    held = [-(-x // P) for x in ctx]
    need = [-(-(x + max(n, 0)) // P) - h if n >= 0 else 0 for n, x, h in zip(new, ctx, held)]
    stride = max(1, max(h + w for h, w in zip(held, need)))
    spare = sum(need) // 2 if c["short"] else sum(need) + 64   # short: not enough for all
    pool = sum(held) + spare
    perm = torch.randperm(max(pool, 1), generator=gen, device=dev).to(torch.int32)
    cols = torch.arange(stride, device=dev)
    at = torch.tensor(_starts(held)[:-1], device=dev)[:, None] + cols
    inside = cols < torch.tensor(held, device=dev)[:, None]
    table = torch.where(inside, perm[at.clamp_(max=max(pool, 1) - 1)], -1).to(torch.int32)
    free = torch.full((max(pool, 1),), -1, dtype=torch.int32, device=dev)
    free[:spare] = perm[sum(held):sum(held) + spare]
    i32 = dict(dtype=torch.int32, device=dev)
    return dict(case=c, op="pages", block_table=table, free_pages=free,
                free_count=torch.tensor([spare], **i32), seq_len=torch.tensor(ctx, **i32),
                new_tokens=torch.tensor(new, **i32),
                released=torch.tensor([_gone(c, x) for x in ctx], **i32) if c["window"] else None,
                slots=sum(max(n, 0) for n in new) + 5)


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    if c["op"] == "pages":
        return _prepare_pages(c, seed, gen, dev)
    new, ctx = _lengths(c)
    seq = [a + b for a, b in zip(new, ctx)]
    table, first_row, rows = _placement(c, seq, gen, dev)
    i32 = dict(dtype=torch.int32, device=dev)
    s = dict(case=c, op=c["op"], new=new, ctx=ctx, rows=rows, block_table=table,
             kv_start_idx=first_row, q_start=torch.tensor(_starts(new), **i32),
             seq_len=torch.tensor(seq, **i32), positions=torch.tensor(ctx, **i32))
    total, t16 = sum(new), T16[c["q"]]
    s["q"] = _normal((total, c["qh"], c["d"]), t16, gen, dev)
    if c["op"] != "append":
        s["k"], s["k_scale"], s["k_scales"] = _filled(c, rows, gen, dev)
        s["v"], s["v_scale"], s["v_scales"] = _filled(c, rows, gen, dev)
        return s
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
    s["q_norm"] = s["k_norm"] = s["rotary"] = s["axis_positions"] = s["pair_axes"] = None
    if c["norm"] != "none":
        t = torch.float32 if c["norm"] == "f32" else t16
        s["q_norm"], s["k_norm"] = (
            (1.0 + 0.2 * torch.randn(c["d"], generator=gen, device=dev)).to(t) for _ in range(2))
    if c["rot"]:
        reach = max(seq)
        if c["axes"] != "none":
            s["axis_positions"], reach = _axis_positions(total, seed, dev)
            s["pair_axes"] = _pair_axes(c)
        s["rotary"] = _table64(c["rot"], reach, dev).float()
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _new_rows(s):
    """Cache rows of every packed token, and their positions."""
    seq = torch.repeat_interleave(torch.arange(len(s["new"]), device="cuda"),
                                  s["q_start"][1:] - s["q_start"][:-1], output_size=sum(s["new"]))
    pos = s["positions"][seq] + torch.arange(len(seq), device="cuda") - s["q_start"][seq]
    return _rows_at(s, seq, pos), pos


def _rows_at(s, seq, pos):
    """Cache rows of the tokens at `pos` of the sequences `seq`."""
    if s["block_table"] is None:
        return s["kv_start_idx"][seq].long() + pos
    P = s["case"]["page"]
    return s["block_table"][seq, pos // P].long() * P + pos % P


def _values(s, which, rows, dtype):
    """The values of cache rows, in `dtype`: [..., KVH, D]."""
    c = s["case"]
    x = s[which].view(-1, c["kvh"], c["d"])[rows]
    if c["kv"] == "e4m3":
        x = x.view(torch.float8_e4m3fn)
    x = x.to(dtype)
    if c["kv"] in QMAX:
        scale, fine = s[which + "_scale"], s[which + "_scales"]
        if c["scales"] == "head":
            x = x * (scale * fine)[:, None]
        elif c["scales"] == "token":
            x = x * (scale * fine[rows])[..., None]
        else:
            x = x * scale
    return x


def _plain_decode(s):
    """Every sequence's visible keys gathered side by side: the first tokens,
    then those of the window."""
    c = s["case"]
    B, KVH, G, D = c["batch"], c["kvh"], c["qh"] // c["kvh"], c["d"]
    T = s["seq_len"].long()[:, None]
    longest = max(n + x for n, x in zip(s["new"], s["ctx"]))
    first, near = min(c["sinks"], longest), min(c["window"], longest)
    i = torch.arange(first + near, device="cuda")[None, :]
    start = (T - c["window"]).clamp(min=0)
    t = torch.where(i < first, i, start + i - first)
    seen = torch.where(i < first, i < T, (t < T) & (t >= c["sinks"]))
    rows = _rows_at(s, torch.arange(B, device="cuda")[:, None], torch.minimum(t, T - 1))
    k, v = (_values(s, w, rows, torch.float32) for w in "kv")
    q = s["q"].float().view(B, KVH, G, D)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * D ** -0.5   # [B, KVH, G, keys]
    score.masked_fill_(~seen[:, None, None, :], -math.inf)
    m = score.amax(-1, keepdim=True)
    score.sub_(m).exp_()
    z = score.sum(-1, keepdim=True)
    o = torch.matmul(score, v.transpose(1, 2)) / z
    return {"out": o.reshape(B, c["qh"], D).to(s["q"].dtype),
            "lse": (m + z.log()).reshape(B, c["qh"])}


def _plain_prefill(s):
    c = s["case"]
    out, lse, at = torch.empty_like(s["q"]), [], 0
    KVH, G, D, W, S = c["kvh"], c["qh"] // c["kvh"], c["d"], c["window"], c["sinks"]
    for b, (n, ctx) in enumerate(zip(s["new"], s["ctx"])):
        # the keys that some token sees
        near = max(0, ctx - W + 1)
        t = torch.arange(n + ctx, device="cuda") if near <= S else torch.cat(
            [torch.arange(S, device="cuda"), torch.arange(near, n + ctx, device="cuda")])
        rows = _rows_at(s, b, t)
        k, v = (_values(s, w, rows, torch.float32).transpose(0, 1) for w in "kv")
        q = s["q"][at:at + n].float().view(n, KVH, G, D).permute(1, 2, 0, 3).reshape(KVH, G * n, D)
        score = (torch.bmm(q, k.transpose(1, 2)) * D ** -0.5).view(KVH, G, n, len(t))
        p = ctx + torch.arange(n, device="cuda")[:, None]
        score.masked_fill_((t > p) | ((t <= p - W) & (t >= S)), -math.inf)
        m = score.amax(-1, keepdim=True)
        score.sub_(m).exp_()
        z = score.sum(-1, keepdim=True)
        o = torch.bmm(score.view(KVH, G * n, len(t)), v).view(KVH, G, n, D) / z
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, c["qh"], D)
        lse.append((m + z.log()).squeeze(-1).permute(2, 0, 1).reshape(n, c["qh"]))
        at += n
    return {"out": out, "lse": torch.cat(lse)}


def _f32(x):
    return torch.full((), x, dtype=torch.float32, device="cuda")


def _normed(x, w):
    """x: [tokens, heads, D] in 32 bits; sums of squares in 64, since 8-bit
    codes are whole numbers and a value next to a border is either of two."""
    mean = x.double().square().mean(-1, keepdim=True).float()
    return x * (1.0 / (mean + _f32(EPS)).sqrt()) * w.float()


def _rotate(x, cos, sin, rot, pairs):
    """x: [tokens, heads, D] in 32 bits; the first `rot` dims of every head turned."""
    cos, sin = cos[:, None, :], sin[:, None, :]
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


def _plain_append(s):
    c = s["case"]
    rows, pos = _new_rows(s)
    q, k = s["q"].float(), s["k_new"].float()
    if c["norm"] != "none":
        q, k = _normed(q, s["q_norm"]), _normed(k, s["k_norm"])
    if c["rot"]:
        half = c["rot"] // 2
        if c["axes"] == "none":
            cos, sin = s["rotary"][pos].split(half, dim=1)
        else:   # [tokens, pairs]: each pair's own position
            axis = torch.tensor(s["pair_axes"], device="cuda")
            p = s["axis_positions"].long()[axis].T
            pair = torch.arange(half, device="cuda")
            cos, sin = s["rotary"][p, pair], s["rotary"][p, pair + half]
        q = _rotate(q, cos, sin, c["rot"], c["pairs"])
        k = _rotate(k, cos, sin, c["rot"], c["pairs"])
    res = {"q": q.to(s["q"].dtype)}
    for w, x in (("k", k), ("v", s["v_new"].float())):
        cache = s[w].view(-1, c["kvh"], c["d"])
        res[w] = s[w]
        if c["kv"] not in QMAX:
            cache[rows] = x.to(cache.dtype)
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
    return res


def _plain_pages(s):
    """Page bookkeeping of one step in whole-table operations."""
    c, table, free = s["case"], s["block_table"], s["free_pages"]
    P, W, S = c["page"], c["window"], c["sinks"]
    B, stride = table.shape
    L, n = s["seq_len"].long(), s["new_tokens"].long()
    count = s["free_count"].long()
    held, ended = (L + P - 1) // P, n < 0
    cols = torch.arange(stride, device="cuda")[None, :]
    # columns that go back: an ended request's, and those that no later token sees
    keep, gone = -(-S // P), torch.zeros_like(L)
    if W:
        gone = s["released"].long().clamp(min=keep)
        dead = torch.maximum(gone, torch.minimum(((L - W + 1).clamp(min=0) // P), held))
        back = torch.where(ended[:, None], (cols < held[:, None]) &
                           ((cols < keep) | (cols >= gone[:, None])),
                           (cols >= gone[:, None]) & (cols < dead[:, None]))
    else:
        back = ended[:, None] & (cols < held[:, None])
    order = torch.cumsum(back.flatten().long(), 0)
    to = torch.where(back.flatten(), count + order - 1, len(free))   # (len(free): nowhere)
    stack = torch.cat([free, free.new_zeros(1)])
    stack[to] = table.flatten()
    stack = stack[:-1]
    avail = count + order[-1]
    # pages for the growing requests, in order, while they last
    need = torch.where(ended, 0, (L + n.clamp(min=0) + P - 1) // P - held)
    upto = torch.cumsum(need, 0)
    granted = ~ended & ((need == 0) | (upto <= avail))
    need = torch.where(granted, need, 0)
    first = upto - need
    take = (cols >= held[:, None]) & (cols < (held + need)[:, None])
    at = (avail - 1 - first[:, None] - (cols - held[:, None])).clamp(0, len(free) - 1)
    table.copy_(torch.where(take, stack[at], table))
    free.copy_(stack)
    # the packed tokens
    grow = n.clamp(min=0)
    q_start = torch.cat([grow.new_zeros(1), torch.cumsum(grow, 0)])
    i = torch.arange(s["slots"], device="cuda")
    b = torch.searchsorted(q_start[1:], i, right=True)
    inside = b < B
    b = b.clamp(max=B - 1)
    pos = L[b] + i - q_start[b]
    page = table[b, (pos // P).clamp(max=stride - 1)].long()
    res = {"q_start": q_start.int(), "positions": torch.where(granted, L, -1).int(),
           "seq_len": torch.where(ended, 0, torch.where(granted, L + n, L)).int(),
           "free_count": (avail - need.sum()).int(), "block_table": table, "free_pages": free,
           "slots": torch.where(inside & granted[b], page * P + pos % P, -1)}
    if W:
        res["released"] = torch.where(ended, 0, dead).int()
    return res


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _own(s):
    import flash_decoding_attention_gb300 as fda
    c = s["case"]
    if s["op"] == "pages":
        if "workspace" not in s:   # a serving program keeps it from step to step
            s["workspace"] = fda.alloc_page_workspace(c["batch"])
        step = fda.assign_pages(s["block_table"], s["seq_len"], s["new_tokens"], s["free_pages"],
                                s["free_count"], c["page"], num_slots=s["slots"],
                                window=c["window"] or None,
                                sinks=c["sinks"] if c["window"] else 0,
                                released=s["released"], workspace=s["workspace"])
        res = {"q_start": step.q_start, "positions": step.positions, "seq_len": step.seq_len,
               "free_count": step.free_count, "block_table": s["block_table"],
               "free_pages": s["free_pages"], "slots": step.slots}
        if c["window"]:
            res["released"] = step.released
        return res
    kw = dict(kv_start_idx=s["kv_start_idx"], block_table=s["block_table"], k_scale=s["k_scale"],
              v_scale=s["v_scale"], k_scales=s["k_scales"], v_scales=s["v_scales"])
    if s["op"] == "decode":
        if "workspace" not in s:
            s["workspace"] = fda.alloc_workspace(c["batch"], c["qh"], c["kvh"], c["d"])
        out, lse = fda.decode_attention(s["q"], s["k"], s["v"], s["seq_len"], window=c["window"],
                                        sinks=c["sinks"], workspace=s["workspace"], **kw)
        return {"out": out, "lse": lse}
    if "workspace" not in s:
        s["workspace"] = fda.alloc_prefill_workspace(c["d"])
    kw["workspace"] = s["workspace"]
    if s["op"] == "prefill":
        out, lse = fda.prefill_attention(s["q"], s["k"], s["v"], s["q_start"], s["seq_len"],
                                         window=c["window"], sinks=c["sinks"], **kw)
        return {"out": out, "lse": lse}
    q = fda.append_kv(s["k_new"], s["v_new"], s["k"], s["v"], s["q_start"], s["positions"],
                      q=s["q"], rotary=s["rotary"], interleaved=c["pairs"] == "interleaved",
                      q_norm=s["q_norm"], k_norm=s["k_norm"], norm_eps=EPS,
                      axis_positions=s["axis_positions"], pair_axes=s["pair_axes"], **kw)
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
    if s["op"] == "pages":
        return _plain_pages(s)
    if s["op"] == "decode":
        return _plain_decode(s)
    return _plain_prefill(s) if s["op"] == "prefill" else _plain_append(s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _seen(n, ctx, W, S):
    """(query, key) pairs of n tokens behind ctx others, and keys that one of them sees."""
    p = np.arange(ctx, ctx + n, dtype=np.int64)
    near = np.maximum(0, p - W + 1)
    pairs = int((p + 1 - near + np.minimum(near, S)).sum())
    lo = int(near[0])
    return pairs, n + ctx - lo + min(lo, S)


def work(case):
    c = case
    new, ctx = _lengths(c)
    if c["op"] == "pages":
        P, W = c["page"], c["window"]
        grow = sum(max(n, 0) for n in new)
        pages = sum(-(-(x + n) // P) - -(-x // P) for n, x in zip(new, ctx) if n >= 0)
        back = 0
        for n, x in zip(new, ctx):
            held, keep, gone = -(-x // P), -(-c["sinks"] // P), _gone(c, x) if W else 0
            if n < 0:
                back += min(keep, held) + max(0, held - gone) if W else held
            elif W:
                back += max(0, min(max(0, x - W + 1) // P, held) - gone)
        moved = grow + 2 * pages + 2 * back
        return {"bytes": c["batch"] * (20 + (8 if W else 0)) + 8 * grow + 8 * (pages + back),
                "flops": moved + 8 * c["batch"]}
    total = sum(new)
    code = 1 if c["kv"] in QMAX else 2
    per_row = 2 * c["kvh"] * (c["d"] * code + (4 if c["scales"] == "token" else 0))
    if c["op"] == "append":
        rows = total * 2 * (c["qh"] + 2 * c["kvh"]) * c["d"]
        back = total * (2 * c["qh"] * c["d"] + per_row)
        turned = 4 * c["rot"] * len({p for n, x in zip(new, ctx) for p in range(x, x + n)}) \
            if c["axes"] == "none" else 12 * total
        norm = 5 * total * (c["qh"] + c["kvh"]) * c["d"] if c["norm"] != "none" else 0
        return {"bytes": rows + back + turned,
                "flops": total * (3 * (c["qh"] + c["kvh"]) * c["rot"] + 2 * c["kvh"] * c["d"]) + norm}
    seen = [_seen(n, x, c["window"], c["sinks"]) for n, x in zip(new, ctx)]
    return {"bytes": sum(k for _, k in seen) * per_row + total * c["qh"] * (4 * c["d"] + 4),
            "flops": 4 * sum(p for p, _ in seen) * c["qh"] * c["d"]}


# ---------------------------------------------------------------------------
# the same results from their definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_rows(s, b, tokens):
    """Cache row of each of these tokens of sequence b, counted out on the host."""
    if s["block_table"] is None:
        first = int(s["kv_start_idx"][b])
        return torch.tensor([first + t for t in tokens], device="cuda")
    P, pages = s["case"]["page"], s["block_table"][b].tolist()
    return torch.tensor([pages[t // P] * P + t % P for t in tokens], device="cuda")


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


def _exact_attention(c, s):
    G, W, S = c["qh"] // c["kvh"], c["window"], c["sinks"]
    outs, lses, at = [], [], 0
    for b, (n, ctx) in enumerate(zip(s["new"], s["ctx"])):
        q = s["q"][at:at + n].double()
        o = torch.empty_like(q)
        l = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
        for lo in range(0, n, 1024):   # some queries at a time
            hi = min(n, lo + 1024)
            tokens = [t for t in range(ctx + hi) if t < S or t > ctx + lo - W]
            rows = _exact_rows(s, b, tokens)
            k, v = _exact_values(s, "k", rows), _exact_values(s, "v", rows)
            t = torch.tensor(tokens, device="cuda")[None, :]
            p = (ctx + torch.arange(lo, hi, device="cuda"))[:, None]
            sees = (t <= p) & ((p - t < W) | (t < S))
            for h in range(c["kvh"]):
                e = torch.einsum("qgd,kd->gqk", q[lo:hi, h * G:(h + 1) * G], k[:, h]) / math.sqrt(c["d"])
                e = torch.where(sees, e, -math.inf)
                z = torch.logsumexp(e, 2)
                l[lo:hi, h * G:(h + 1) * G] = z.T
                o[lo:hi, h * G:(h + 1) * G] = torch.einsum("gqk,kd->qgd", torch.exp(e - z[..., None]), v[:, h])
        outs.append(o)
        lses.append(l)
        at += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def exact(case, seed):
    c = case
    if c["op"] == "pages":   # whole numbers all
        return None
    s = prepare(case, seed)
    if c["op"] != "append":
        return _exact_attention(c, s)
    rows, pos = [], []
    for b, (n, ctx) in enumerate(zip(s["new"], s["ctx"])):
        rows.append(_exact_rows(s, b, range(ctx, ctx + n)))
        pos += range(ctx, ctx + n)
    rows = torch.cat(rows)
    q, k, v = s["q"].double(), s["k_new"].double(), s["v_new"].double()
    if c["norm"] != "none":
        eps = float(np.float32(EPS))
        q = q * s["q_norm"].double() / torch.sqrt((q * q).sum(-1, keepdim=True) / c["d"] + eps)
        k = k * s["k_norm"].double() / torch.sqrt((k * k).sum(-1, keepdim=True) / c["d"] + eps)
    if c["rot"]:
        half, t = c["rot"] // 2, s["rotary"].double()
        turn = torch.empty((len(pos), half), dtype=torch.complex128, device="cuda")
        for i in range(half):
            p = torch.tensor(pos, device="cuda") if c["axes"] == "none" else \
                s["axis_positions"][s["pair_axes"][i]].long()
            turn[:, i] = torch.complex(t[p, i], t[p, half + i])
        turn = turn[:, None, :]
        for x in (q, k):
            if c["pairs"] == "half":
                z = torch.complex(x[..., :half].contiguous(), x[..., half:c["rot"]].contiguous()) * turn
                x[..., :half], x[..., half:c["rot"]] = z.real, z.imag
            else:
                z = torch.complex(x[..., 0:c["rot"]:2].contiguous(),
                                  x[..., 1:c["rot"]:2].contiguous()) * turn
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
