"""Plain 64-bit statement of attention with a sliding window and first tokens,
and batches whose hidden rows and pages hold the worst that may lie there."""
from __future__ import annotations

import math

import numpy as np
import torch

import prompt_ref as ref


def sees(pos, window, sinks):
    """Tokens that the query at `pos` sees, ascending."""
    if pos < 0:
        return torch.zeros(0, dtype=torch.long)
    t = torch.arange(pos + 1)
    return t[(t > pos - window) | (t < sinks)]


def attention(filled, q, qh, scale, window, sinks):
    """(out, lse) of packed queries [tokens, qh, d]; rows of nobody are NaN."""
    bt = filled.batch
    group = qh // bt.kvh
    out = torch.full(q.shape, float("nan"), dtype=torch.float64)
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float64)
    for b, (n, T) in enumerate(zip(bt.new, bt.seq)):
        if n == 0:
            continue
        rows = bt.rows_of(b, 0, T)
        i = int(bt.q_start[b])
        pos = (bt.ctx[b] + torch.arange(n))[:, None]
        t = torch.arange(T)[None, :]
        seen = (t <= pos) & ((t > pos - window) | (t < sinks))   # [n, T]
        used = seen.any(0)
        rows, seen = rows[used], seen[:, used]
        for h in range(qh):
            k, v = filled.val["k"][rows, h // group], filled.val["v"][rows, h // group]
            s = q[i:i + n, h].double() @ k.T * scale
            s = torch.where(seen, s, torch.tensor(-math.inf, dtype=torch.float64))
            z = torch.logsumexp(s, -1) if len(rows) else torch.full((n,), -math.inf,
                                                                    dtype=torch.float64)
            w = torch.exp(s - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
            w = torch.where(seen, w, torch.zeros_like(w))
            lse[i:i + n, h] = z
            # a value reaches the rows that see it (0 * NaN is no reading of it)
            fine = torch.isfinite(v)
            o = w @ torch.where(fine, v, torch.zeros_like(v)) if len(rows) else \
                torch.zeros((n, bt.d), dtype=torch.float64)
            for r, d in (~fine).nonzero().tolist():
                o[seen[:, r], d] += w[seen[:, r], r] * v[r, d]
            out[i:i + n, h] = o
    return out, lse


def hide(filled, window, sinks):
    """What no query of the batch sees: rows become NaN (or the worst codes) with
    NaN scales, and the table entries of pages without a visible token wrong page
    ids, as of pages given away.  Call it before the statement reads `val`."""
    bt = filled.batch
    cut = 0
    for b, (n, T) in enumerate(zip(bt.new, bt.seq)):
        seen = torch.zeros(T, dtype=torch.bool)
        for p in range(max(0, T - n), T):
            seen[sees(p, window, sinks)] = True
        gone = (~seen).nonzero().flatten().tolist()
        for t in gone:
            row = bt.row(b, t)
            for w in "kv":
                c = filled.kw[w + "_cache"].view(bt.rows, bt.kvh, bt.d)
                c[row] = ref.poison(bt.kv, (bt.kvh, bt.d))
                filled.val[w][row] = float("nan")
                if filled.scales == "token":
                    filled.kw[w + "_scales"][row] = float("nan")
        if bt.page:
            for c in range(-(-T // bt.page)):
                if not seen[c * bt.page:(c + 1) * bt.page].any():
                    bt.block_table[b, c] = [-1, 10 ** 9, -(1 << 31)][c % 3]
                    cut += 1
        del gone
    return cut


def compare(bt, out, lse, want, wlse, x16, label="", fill=7.0):
    """Rows of nobody hold `fill`; the others are the statement's."""
    mine = torch.zeros(out.shape[0], dtype=torch.bool)
    for b, n in enumerate(bt.new):
        mine[int(bt.q_start[b]):int(bt.q_start[b]) + n] = True
    assert torch.all(out[~mine] == fill) and torch.all(lse[~mine] == fill), label
    out, lse, want, wlse = out[mine], lse[mine], want[mine], wlse[mine]
    empty = wlse == -math.inf
    assert torch.equal(lse == -math.inf, empty) and torch.all(out[empty] == 0), label
    out, lse, want, wlse = out[~empty], lse[~empty], want[~empty], wlse[~empty]
    if not len(out):
        return
    # A probability and the output are each rounded once to 16 bits: half a
    # step, eps / 2, of the value.  The probabilities' errors reach the output
    # weighted by v: at most eps / 2 * max |v|, with N(0, 1) draws of these
    # sizes below 5.5; the output's own eps / 2 * |out|.  fp32 products, sums
    # and ex2 add a few 2^-22 of the same magnitudes.
    eps = torch.finfo(ref.T16[x16]).eps
    tol = (eps / 2 + 2.0 ** -18) * 5.5 + (eps / 2) * want.abs()
    assert torch.all((out - want).abs() <= tol), (label, float(((out - want).abs() - tol).max()))
    # scores up to about 40 in fp32 (128 products), and ex2 / lg2
    assert float((lse - wlse).abs().max()) <= 1e-4 * max(1.0, float(wlse.abs().max())), label
    rel = float(torch.linalg.norm(out - want) / torch.linalg.norm(want))
    assert rel <= eps, (label, rel)     # two independent roundings: sqrt(2) eps / sqrt(12) rms
