"""GPU tests of the page bookkeeping's lengths for the attention: what refused,
idle and ended sequences of a sliding-window step leave to it."""
import math

import numpy as np
import pytest
import torch

from gpu_util import lib
from test_gpu_pages import DEV, I32, State

pytestmark = pytest.mark.gpu


def _lengths(got, new):
    """The statement: the new length of a served sequence with new tokens."""
    return [s if p >= 0 and n > 0 else 0
            for s, p, n in zip(got.seq_len.tolist(), got.positions.tolist(), new)]


@pytest.mark.parametrize("B", [5, 300, 1024, 2500])
@pytest.mark.parametrize("window", [0, 40])
def test_lengths_of_many_kinds(B, window):
    """Both forms of the call; without a window only where an array is given."""
    rng = np.random.default_rng(B + window)
    page, width = 16, 6
    s = State(rng, B, width, max(2, B * width // 3), page, window, 20 if window else 0)
    for k in range(5):
        new = rng.choice([-1, 0, 1, 1, 2, 17, 33], B)
        new = [int(min(n, width * page - L)) if n > 0 else int(n) for n, L in zip(new, s.seq)]
        own = torch.full((B,), 77, **I32) if k % 2 or not window else None
        got, _ = s.step(new, [None, sum(max(n, 0) for n in new)][k % 2],
                        **({} if own is None else dict(attend_len=own)))
        assert own is None or got.attend_len is own
        assert got.attend_len.tolist() == _lengths(got, new)
        assert any(got.attend_len.tolist()) or B == 5
        q_start, _, seq, _, _, _ = got           # the tuple's entries are the arrays of the state
        assert q_start is got.q_start and seq is got.seq_len
    if not window:
        assert s.step([0] * B)[0].attend_len is None


QH, KVH, P, W = 8, 2, 4, 21


def _filled(st, pool, D, seed):
    """Caches whose pages in use hold numbers and whose others hold NaN."""
    g = torch.Generator().manual_seed(seed)
    kv = torch.randn((2, pool, P, KVH, D), generator=g).clamp(-5.5, 5.5).half()
    used = torch.zeros(pool, dtype=torch.bool)
    for row, L in zip(st.table, st.seq):
        used[row[:-(-L // P)]] = True
    kv[:, ~used] = float("nan")
    return kv


def _attended(keys, vals, q, pos, sinks):
    """64 bits: queries at `pos` over keys [T, KVH, D]."""
    t = torch.arange(len(keys))[None, :]
    seen = (t <= pos[:, None]) & ((t > pos[:, None] - W) | (t < sinks))
    k, v = (x.double().repeat_interleave(QH // KVH, 1) for x in (keys, vals))
    hidden = ~seen.any(0)
    k[hidden], v[hidden] = 0, 0                       # (NaN where nobody looks)
    s = torch.einsum("qhd,khd->qhk", q.double(), k) / q.shape[-1] ** 0.5
    s = s.masked_fill(~seen[:, None, :], -math.inf)
    return torch.einsum("qhk,khd->qhd", s.softmax(-1), v), s.logsumexp(-1)


# (cached, new) of a step's sequences.  Some are served with a page or without,
# some refused for want of pages, one idles, one has ended.  Of 36 and 40 cached
# tokens the column that ends at L - W + 1 goes back in this step; a query at
# L - 1 sees its last token.
PREFILL = [(22, 7), (36, 25), (40, 0), (43, 1), (9, -1)]
DECODE = [(4, 1), (8, 1), (12, 1), (36, 1), (40, 0), (30, 1)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sinks", [0, 5])
@pytest.mark.parametrize("decode", [False, True])
def test_a_refused_sequence_behind_a_window(decode, sinks, D):
    """Pages that a step gives away are not used by its attention, whoever's they
    were: their entries are overwritten and their rows hold NaN; every row of a
    served sequence is right, every other one is empty, nothing is recorded."""
    fda = lib()
    rng = np.random.default_rng(3)
    ctx, new = [list(x) for x in zip(*(DECODE if decode else PREFILL))]
    held = sum(-(-x // P) for x in ctx)
    width, pool = 20, held
    st = State(rng, len(ctx), width, pool, P, W, sinks, lens=list(ctx))
    keep = -(-sinks // P)
    # as the steps before left it: what a token at L - 1 does not see is gone
    st.released = [max(keep, max(0, x - W) // P) for x in ctx]
    st.d_released = torch.tensor(st.released, **I32)
    table0 = [list(r) for r in st.table]
    kv = _filled(st, pool, D, 1)
    kc, vc = kv[0].to(DEV), kv[1].to(DEV)
    n = sum(max(x, 0) for x in new)
    before = list(st.released)
    got, errors = st.step(new, n)
    assert not errors
    pos = got.positions.tolist()
    gone = [(b, c) for b in range(len(ctx)) for c in range(max(keep, before[b]), st.released[b])]
    assert {b for b, _ in gone} == {ctx.index(36), ctx.index(40)}
    refused = [b for b in range(len(ctx)) if new[b] > 0 and pos[b] < 0]
    served = [b for b in range(len(ctx)) if new[b] > 0 and pos[b] >= 0]
    assert ctx.index(36) in refused and len(served) >= 2
    assert got.attend_len.tolist() == _lengths(got, new)
    # entries of everything that is gone: overwritten (their pages may belong to
    # another sequence by now, or hold NaN on the stack)
    for b in range(len(ctx)):
        for c in range(keep, max(keep, st.released[b])):
            st.table[b][c] = 10 ** 6 if c % 2 else -3
    table = torch.tensor(st.table, **I32)
    for page in st.free[:st.count]:
        kc[page] = float("nan")
        vc[page] = float("nan")
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn((n, h, D), generator=g).clamp(-5.5, 5.5).half() for h in (QH, KVH, KVH))
    ws, wsd = fda.alloc_prefill_workspace(D), fda.alloc_workspace(len(ctx), QH, KVH, D)
    if decode:
        fda.append_kv(k.to(DEV), v.to(DEV), kc, vc, got.q_start, got.positions, workspace=ws,
                      block_table=table)
        # one query a sequence of the batch, the idle one's too
        qb = torch.randn((len(ctx), QH, D), generator=g).half()
        qb[[b for b in range(len(ctx)) if new[b] == 1]] = q
        out, lse = fda.decode_attention(qb.to(DEV), kc, vc, got.attend_len, block_table=table,
                                        window=W, sinks=sinks, workspace=wsd)
        rows_of = [slice(b, b + 1) for b in range(len(ctx))]
    else:
        qb = q
        out, lse = fda.prefill_attention(q.to(DEV), kc, vc, got.q_start, got.attend_len,
                                         k_new=k.to(DEV), v_new=v.to(DEV),
                                         positions=got.positions, block_table=table, window=W,
                                         sinks=sinks, workspace=ws)
        starts = got.q_start.tolist()
        rows_of = [slice(a, z) for a, z in zip(starts, starts[1:])]
    torch.cuda.synchronize()
    for w in (ws, wsd):
        assert fda.fd_check_device_error(w)[0] == fda.FD_OK
    out, lse = out.double().cpu(), lse.double().cpu()
    starts = got.q_start.tolist()
    for b in range(len(ctx)):
        rows = rows_of[b]
        if b not in served:
            assert torch.all(out[rows] == 0) and torch.all(lse[rows] == -math.inf)
            continue
        at = [table0[b][t // P] * P + t % P for t in range(ctx[b])]
        mine = slice(starts[b], starts[b + 1])
        keys = torch.cat([kv[0].view(-1, KVH, D)[at], k[mine]])
        vals = torch.cat([kv[1].view(-1, KVH, D)[at], v[mine]])
        where = torch.arange(ctx[b], ctx[b] + new[b])
        want, wl = _attended(keys, vals, qb[rows], where, sinks)
        # a probability and the output, each half a step of f16 (2^-11); fp32 sums
        tol = (2.0 ** -11 + 2.0 ** -18) * 5.5 + 2.0 ** -11 * want.abs()
        assert torch.all((out[rows] - want).abs() <= tol), b
        assert torch.all((lse[rows] - wl).abs() <= 1e-4 * wl.abs().clamp(min=1)), b
