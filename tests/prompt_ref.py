"""Plain 64-bit statements of the prompt path's operators, for its tests: loops
over sequences and tokens, numpy / torch on the CPU, no code of the library."""
from __future__ import annotations

import math

import numpy as np
import torch

QMAX = {"e4m3": 448.0, "i8": 127.0}
T16 = {"f16": torch.float16, "bf16": torch.bfloat16}


class Batch:
    """A batch of sequences in a cache: lengths, placement and index arrays.

    new[b] packed tokens behind ctx[b] cached ones; ``page`` 0 is a contiguous
    cache with a gap of two rows before every sequence.  ``lead`` packed rows
    lie before the first sequence's tokens and ``tail`` behind the last one's;
    both belong to nobody."""

    def __init__(self, new, ctx, kvh, d, kv, page=0, seed=0, lead=0, tail=0):
        self.new, self.ctx, self.kvh, self.d, self.kv, self.page = new, ctx, kvh, d, kv, page
        rng = np.random.default_rng(seed)
        seq = [max(0, n + c) for n, c in zip(new, ctx)]
        self.seq = seq
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32) + lead
        self.tokens = int(self.q_start[-1]) + tail
        self.block_table = self.kv_start_idx = None
        if page:
            need = [-(-t // page) for t in seq]
            pool = int(sum(need) * 1.3) + 2
            self.rows = pool * page
            perm = rng.permutation(pool).astype(np.int32)
            self.block_table = np.full((len(new), max(need + [1])), 10 ** 9, np.int32)
            at = 0
            for b, n in enumerate(need):
                self.block_table[b, :n] = perm[at:at + n]
                at += n
        else:
            starts, at = [], 2
            for t in seq:
                starts.append(at)
                at += t + 2
            self.rows = at
            self.kv_start_idx = np.array(starts, np.int32)

    def row(self, b, t):
        if self.page:
            return int(self.block_table[b, t // self.page]) * self.page + t % self.page
        return int(self.kv_start_idx[b]) + t

    def rows_of(self, b, lo, hi):
        return torch.tensor([self.row(b, t) for t in range(lo, hi)], dtype=torch.long)

    def shape(self):
        head = (self.rows // self.page, self.page) if self.page else (self.rows,)
        return head + (self.kvh, self.d)

    def index(self, device):
        """The index arrays on the device, as keyword arguments."""
        def t(a):
            return None if a is None else torch.from_numpy(a).to(device)
        return dict(kv_start_idx=t(self.kv_start_idx), block_table=t(self.block_table))


def poison(kv, shape):
    """A cache whose every row is unowned: NaN, or the codes worst to read."""
    if kv == "e4m3":
        return torch.full(shape, 0x7F, dtype=torch.uint8)      # NaN
    if kv == "i8":
        return torch.full(shape, 127, dtype=torch.int8)
    return torch.full(shape, float("nan"), dtype=T16[kv])


def store_type(kv):
    return T16.get(kv) or (torch.uint8 if kv == "e4m3" else torch.int8)


def codes_of(x, kv):
    """fp32 / fp64 values -> stored elements, rounded and clamped."""
    if kv in T16:
        return x.to(T16[kv])
    x = x.clamp(-QMAX[kv], QMAX[kv])
    if kv == "e4m3":
        return x.float().to(torch.float8_e4m3fn).view(torch.uint8)
    return x.round().to(torch.int8)


def value_of(codes, kv):
    return (codes.view(torch.float8_e4m3fn).float() if kv == "e4m3" else codes).double()


class Filled:
    """A batch's caches holding N(0, 1) values of every owned row, poison
    elsewhere; scales per tensor, head or token."""

    def __init__(self, batch, scales="tensor", seed=1):
        g = torch.Generator().manual_seed(seed)
        kv = batch.kv
        self.batch, self.scales = batch, scales
        self.kw = {}
        owned = torch.cat([batch.rows_of(b, 0, t) for b, t in enumerate(batch.seq)] +
                          [torch.zeros(0, dtype=torch.long)])
        self.val = {}
        for w in "kv":
            x = torch.randn((len(owned), batch.kvh, batch.d), generator=g, dtype=torch.float64)
            scale, fine = 1.0, None
            if kv in QMAX:
                scale = float(np.float32(5.0 / QMAX[kv]))
                if scales == "head":
                    fine = torch.rand(batch.kvh, generator=g) + 0.5
                    step = scale * fine.double()[None, :, None]
                elif scales == "token":
                    fine = torch.full((batch.rows, batch.kvh), float("nan"))
                    fine[owned] = torch.rand((len(owned), batch.kvh), generator=g) + 0.5
                    step = scale * fine[owned].double()[:, :, None]
                else:
                    step = scale
                codes = codes_of(x / step, kv)
                x = value_of(codes, kv) * step
            else:
                codes = x.to(T16[kv])
                x = codes.double()
            cache = poison(kv, (batch.rows, batch.kvh, batch.d))
            cache[owned] = codes
            full = torch.full((batch.rows, batch.kvh, batch.d), float("nan"), dtype=torch.float64)
            full[owned] = x
            self.val[w] = full
            self.kw[w + "_cache"] = cache.view(batch.shape())
            self.kw[w + "_scale"] = scale
            self.kw[w + "_scales"] = fine

    def device(self, dev):
        return {k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in self.kw.items()}


def attention(filled, q, qh, softmax_scale, causal_limit=None):
    """(out, lse) in 64 bits for packed queries [tokens, qh, d]; rows of nobody
    are NaN."""
    bt = filled.batch
    group = qh // bt.kvh
    out = torch.full(q.shape, float("nan"), dtype=torch.float64)
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float64)
    for b in range(len(bt.new)):
        for j in range(bt.new[b]):
            i = int(bt.q_start[b]) + j
            seen = bt.seq[b] - (bt.new[b] - 1 - j)
            if seen <= 0:
                out[i] = 0.0
                lse[i] = -math.inf
                continue
            rows = bt.rows_of(b, 0, seen)
            for h in range(bt.kvh):
                k, v = filled.val["k"][rows, h], filled.val["v"][rows, h]
                s = q[i, h * group:(h + 1) * group].double() @ k.T * softmax_scale
                z = torch.logsumexp(s, -1)
                lse[i, h * group:(h + 1) * group] = z
                out[i, h * group:(h + 1) * group] = torch.exp(s - z[:, None]) @ v
    return out, lse


def attention_blocks(filled, q, qh, softmax_scale):
    """The same as `attention`, a sequence at a time in matrix form (for
    batches of many tokens)."""
    bt = filled.batch
    group = qh // bt.kvh
    out = torch.full(q.shape, float("nan"), dtype=torch.float64)
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float64)
    for b in range(len(bt.new)):
        n, T = bt.new[b], bt.seq[b]
        i = int(bt.q_start[b])
        if n == 0:
            continue
        rows = bt.rows_of(b, 0, T)
        seen = torch.arange(T)[None, :] < (T - n + 1 + torch.arange(n))[:, None]   # [n, T]
        for h in range(qh):
            k, v = filled.val["k"][rows, h // group], filled.val["v"][rows, h // group]
            s = q[i:i + n, h].double() @ k.T * softmax_scale
            s = torch.where(seen, s, torch.tensor(-math.inf, dtype=torch.float64))
            z = torch.logsumexp(s, -1) if T else torch.full((n,), -math.inf, dtype=torch.float64)
            w = torch.exp(s - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
            lse[i:i + n, h] = z
            out[i:i + n, h] = torch.where(seen, w, torch.zeros_like(w)) @ v if T else 0.0
    return out, lse


def table(positions, rot, theta, scaling="none", factor=1.0, original=0.0, low=1.0, high=32.0,
          amplitude=1.0):
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        g = np.clip((original * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
        f = g * f + (1.0 - g) * f / factor
    a = np.arange(positions, dtype=np.float64)[:, None] * f[None, :]
    return amplitude * np.concatenate([np.cos(a), np.sin(a)], axis=1)


def rotate(x, tab, pos, rot, interleaved, dtype):
    """[tokens, heads, d] turned in `dtype` arithmetic, one rounding per product
    and sum (torch has no contraction between separate operations)."""
    x = x.to(dtype).clone()
    c = tab[pos][:, None, :rot // 2].to(dtype)
    s = tab[pos][:, None, rot // 2:].to(dtype)
    if interleaved:
        a, b = x[..., 0:rot:2].clone(), x[..., 1:rot:2].clone()
        x[..., 0:rot:2], x[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2].clone(), x[..., rot // 2:rot].clone()
        x[..., :rot // 2], x[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return x


def quantise(x, kv, scale, fine, kind):
    """fp32 rows [tokens, kvh, d] -> (codes, per-token scales or None), each
    product and quotient one fp32 operation."""
    if kv in T16:
        return x.to(T16[kv]), None
    s = torch.tensor(scale, dtype=torch.float32)
    tok = None
    if kind == "head":
        s = (s * fine)[None, :, None]
    elif kind == "token":
        amax = x.abs().amax(-1)
        tok = torch.where(amax > 0, amax / (torch.tensor(QMAX[kv]) * s), torch.tensor(1.0))
        s = (s * tok)[:, :, None]
    return codes_of(x / s, kv), tok
