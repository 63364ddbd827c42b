"""GPU tests of the page bookkeeping against a plain one on the host, and of a
sliding-window model's serving steps through all of their calls."""
import math

import numpy as np
import pytest
import torch

import pages_ref
import prompt_ref as ref
import window_ref as wref
from gpu_util import lib
from test_gpu_norms import axes_of, normed, turned

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = dict(dtype=torch.int32, device=DEV)


class State:
    """A page state on the host and its copy on the device."""

    def __init__(self, rng, B, width, pool, page, window=0, sinks=0, lens=None, cap=None):
        self.page, self.window, self.sinks = page, window, sinks
        perm = [int(x) for x in rng.permutation(pool)]
        self.seq = lens or [0] * B
        self.table = []
        for L in self.seq:
            held = min(width, -(-max(L, 0) // page))
            self.table.append([perm.pop() if perm else 0 for _ in range(held)] + [-9] * (width - held))
        self.count = len(perm)
        self.free = perm + [-7] * ((cap or pool) - len(perm))
        self.released = [0] * B
        self.fda = lib()
        self.ws = self.fda.alloc_page_workspace(B)
        self.d_table = torch.tensor(self.table, **I32)
        self.d_free = torch.tensor(self.free, **I32)
        self.d_count = torch.tensor([self.count], **I32)
        self.d_seq = torch.tensor(self.seq, **I32)
        self.d_released = torch.tensor(self.released, **I32) if window else None

    def step(self, new, num_slots=None, in_place=False, **kw):
        """One step on both sides, compared; returns (device step, errors)."""
        want = pages_ref.step(self.table, self.seq, new, self.free, self.count, self.page,
                              self.window, self.sinks, self.released, num_slots)
        over = {}
        if in_place:
            over = dict(seq_len_out=self.d_seq, free_count_out=self.d_count)
            if self.window:
                over["released_out"] = self.d_released
        if num_slots is not None:
            kw["slots"] = torch.full((num_slots,), 5, dtype=torch.int64, device=DEV)
        got = self.fda.assign_pages(self.d_table, self.d_seq, torch.tensor(new, **I32), self.d_free,
                                    self.d_count, self.page, window=self.window or None,
                                    sinks=self.sinks, released=self.d_released, workspace=self.ws,
                                    **over, **kw)
        torch.cuda.synchronize()
        q_start, positions, seq, count, released, slots, errors = want
        assert got.q_start.tolist() == q_start
        assert got.positions.tolist() == positions
        assert got.seq_len.tolist() == seq
        assert got.free_count.tolist() == [count]
        assert self.d_free.tolist() == self.free
        assert self.d_table.tolist() == self.table
        if self.window:
            assert got.released.tolist() == released
            self.released, self.d_released = released, got.released
        if num_slots is not None:
            assert got.slots.tolist() == slots
        st, info = self.fda.fd_check_device_error(self.ws)
        assert (st == self.fda.FD_OK) == (not errors) and (not errors or info in errors)
        self.seq, self.count = seq, count
        self.d_seq, self.d_count = got.seq_len, got.free_count
        return got, errors


@pytest.mark.parametrize("seed", range(20))
def test_steps_of_many_kinds(seed):
    """Requests that start, grow, idle and end over several steps, with and
    without a window, with enough pages or too few: both forms of the call."""
    rng = np.random.default_rng(seed)
    B = [1, 3, 40, 300, 1023, 1024, 1025, 2500][seed % 8]
    page = [1, 2, 16, 64, 256][seed % 5]
    window, sinks = [(0, 0), (1, 0), (40, 4), (100, 33), (7, 70)][(seed // 2) % 5]
    width = int(rng.integers(3, 30))
    pool = max(2, int(B * width * rng.choice([0.2, 0.6, 1.0])))
    s = State(rng, B, width, pool, page, window, sinks)
    for k in range(6):
        new = rng.choice([-1, 0, 1, 1, 1, 2, 17, page, 3 * page], B)
        new = [int(min(n, width * page - L)) if n > 0 else int(n) for n, L in zip(new, s.seq)]
        total = sum(max(n, 0) for n in new)
        slots = [None, total, total + 37][k % 3]
        s.step(new, slots, in_place=k % 2 == 1)
        # a page belongs to one sequence, or lies on the stack
        held = []
        for b, L in enumerate(s.seq):
            n, keep = -(-L // page), -(-sinks // page)
            gone = s.released[b] if window else 0
            held += [s.table[b][c] for c in range(n) if c < keep or c >= gone]
        assert sorted(held + s.free[:s.count]) == list(range(pool))
    s.step([-1] * B)
    assert sorted(s.free[:s.count]) == list(range(pool))


def test_large_steps():
    """Thousands of requests admitted at once, tens of thousands of slots."""
    rng = np.random.default_rng(3)
    s = State(rng, 3000, 40, 50000, 16)
    new = [int(x) for x in rng.integers(0, 600, 3000)]
    s.step(new, sum(new) + 3)
    s.step([-1 if i % 3 else 1 for i in range(3000)], 1000)
    s.step([int(x) for x in rng.integers(0, 40, 3000)])


@pytest.mark.parametrize("slots", [None, 50])
def test_what_is_refused(slots):
    """Too few pages (not recorded), a row or slots that are too short, and a
    table that does not hold its sequence (recorded): nobody else is touched."""
    rng = np.random.default_rng(1)
    s = State(rng, 6, 4, 9, 4, lens=[3, 4, 0, 16, 5, 1])
    assert s.count == 0
    got, errors = s.step([1, 1, 0, -1, 3, 0], slots)       # four pages return, one is wanted
    assert not errors and got.positions.tolist() == [3, 4, 0, -1, 5, 1]
    got, errors = s.step([17, 1, 13, 0, 0, 3], slots)      # a row of 16 tokens; 3 pages left
    assert errors and got.positions.tolist()[0] == -1
    if slots:
        got, errors = s.step([0, 0, 0, 3, 60, 1], slots)   # slots for 50
        assert errors
    s = State(rng, 3, 2, 3, 4, lens=[9, 4, -5])            # nine tokens in two pages of four
    got, errors = s.step([1, 1, 1], slots)
    assert errors and got.positions.tolist()[0] == -1
    s.step([-1, -1, -1], slots)


def test_a_stack_that_overflows_is_recorded():
    rng = np.random.default_rng(1)
    s = State(rng, 3, 4, 8, 2, lens=[8, 6, 2], cap=3)
    got, errors = s.step([-1, 1, -1], 4)
    assert errors and got.free_count.tolist() == [2]
    s.d_count.fill_(9)
    s.count = 9
    got, errors = s.step([0, 0, 2], 4)
    assert errors


def test_far_lengths():
    """Lengths near 2^31 (with a row too short for them), a window longer than
    any sequence, and negative counts."""
    rng = np.random.default_rng(1)
    s = State(rng, 4, 3, 4, 256, (1 << 31) - 1, 1, lens=[5, 0, 700, 2])
    s.step([(1 << 31) - 1, 3, 1, 0])
    s.step([-(1 << 31), 1, 60, -1])
    s.count = -4
    s.d_count.fill_(-4)
    s.step([300, 0, 0, 0], 300)


def test_steps_in_a_graph_and_on_another_stream():
    """A captured step updates lengths, stack and tables in place, replay by
    replay."""
    fda = lib()
    rng = np.random.default_rng(2)
    for many in (False, True):
        s = State(rng, 5, 40, 150, 4, 30, 2)
        slots = torch.zeros(20000 if many else 100, dtype=torch.int64, device=DEV)
        new = torch.zeros(5, **I32)
        kw = dict(window=30, sinks=2, released=s.d_released, seq_len_out=s.d_seq,
                  free_count_out=s.d_count, released_out=s.d_released, slots=slots, workspace=s.ws)
        args = (s.d_table, s.d_seq, new, s.d_free, s.d_count, 4)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        fda.assign_pages(*args, stream=side, **kw)          # nothing new: nothing changes
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = fda.assign_pages(*args, **kw)
        for k in range(12):
            n = [int(x) for x in rng.choice([-1, 0, 1, 1, 3, 20], 5)]
            n = [min(x, 160 - L) if x > 0 else x for x, L in zip(n, s.seq)]
            want = pages_ref.step(s.table, s.seq, n, s.free, s.count, 4, 30, 2, s.released,
                                  len(slots))
            new.copy_(torch.tensor(n, dtype=torch.int32))
            graph.replay()
            torch.cuda.synchronize()
            s.seq, s.count, s.released = want[2], want[3], want[4]
            assert got.q_start.tolist() == want[0] and got.positions.tolist() == want[1]
            assert s.d_seq.tolist() == s.seq and s.d_count.tolist() == [s.count]
            assert s.d_released.tolist() == s.released and slots.tolist() == want[5]
            assert s.d_table.tolist() == s.table and s.d_free.tolist() == s.free


def test_serving_steps_of_a_window_model():
    """Prompts, then chunks beside single tokens, then a decode step, of a model
    with normed heads, three axes and a sliding window over a pool of pages that
    only suffices because those behind the window are used again: every step's
    pages, caches and outputs against the plain statement."""
    fda = lib()
    QH, KVH, D, P, W, S, B = 8, 2, 64, 4, 20, 3, 3
    pool, width = 36, 40
    g = torch.Generator().manual_seed(0)
    rng = np.random.default_rng(0)
    st = State(rng, B, width, pool, P, W, S)
    kc, vc = (torch.full((pool, P, KVH, D), float("nan"), dtype=torch.float16, device=DEV)
              for _ in range(2))
    tab = fda.rotary_table(200, D)
    host_tab = tab.cpu()
    w = [(torch.rand(D, generator=g) + 0.5) for _ in range(2)]
    dw = [x.to(DEV) for x in w]
    axes = axes_of("runs", D)
    ws, wsd = fda.alloc_prefill_workspace(D), fda.alloc_workspace(B, QH, KVH, D)
    keys = [torch.zeros(0, KVH, D) for _ in range(B)]      # what each sequence has cached
    vals = [torch.zeros(0, KVH, D) for _ in range(B)]
    for new in ([30, 7, 0], [1, 16, 25], [12, 1, 1], [1, 1, 1], [25, 1, -1], [1, 1, 9], [1, 1, 1]):
        n = sum(max(x, 0) for x in new)
        q, k, v = (torch.randn((n, h, D), generator=g).half() for h in (QH, KVH, KVH))
        ap = torch.randint(0, 200, (3, n), generator=g, dtype=torch.int32)
        step, _ = st.step(new, n)
        assert all((p >= 0) == (x >= 0) for p, x in zip(step.positions.tolist(), new))
        args = dict(q_norm=dw[0], k_norm=dw[1], rotary=tab, axis_positions=ap.to(DEV),
                    pair_axes=axes, block_table=st.d_table)
        if all(x == 1 for x in new):       # a decode step: rows of the batch
            q2 = fda.append_kv(k.to(DEV), v.to(DEV), kc, vc, step.q_start, step.positions,
                               q=q.to(DEV), workspace=ws, **args)
            out, lse = fda.decode_attention(q2, kc, vc, step.seq_len, block_table=st.d_table,
                                            window=W, sinks=S, workspace=wsd)
        else:
            out, lse = fda.prefill_attention(q.to(DEV), kc, vc, step.q_start, step.seq_len,
                                             k_new=k.to(DEV), v_new=v.to(DEV),
                                             positions=step.positions, window=W, sinks=S,
                                             workspace=ws, **args)
        torch.cuda.synchronize()
        for x in (ws, wsd):
            assert fda.fd_check_device_error(x)[0] == fda.FD_OK
        qn = turned(normed(q.float(), w[0], 1e-6), host_tab, ap, D, False, axes).half().double()
        kn = turned(normed(k.float(), w[1], 1e-6), host_tab, ap, D, False, axes).half().float()
        slots = step.slots.cpu()
        assert torch.equal(kc.cpu().view(-1, KVH, D)[slots].float(), kn)
        assert torch.equal(vc.cpu().view(-1, KVH, D)[slots], v)
        at = 0
        for b in range(B):
            if new[b] < 0:
                keys[b], vals[b] = keys[b][:0], vals[b][:0]
                continue
            rows = slice(at, at + new[b])
            at += new[b]
            keys[b], vals[b] = torch.cat([keys[b], kn[rows]]), torch.cat([vals[b], v[rows].float()])
            T = len(keys[b])
            pos = (T - new[b] + torch.arange(new[b]))[:, None]
            t = torch.arange(T)[None, :]
            seen = (t <= pos) & ((t > pos - W) | (t < S))
            kk = keys[b].double().repeat_interleave(QH // KVH, 1)
            s = torch.einsum("qhd,khd->qhk", qn[rows], kk) / D ** 0.5
            s = s.masked_fill(~seen[:, None, :], -math.inf)
            want = torch.einsum("qhk,khd->qhd", s.softmax(-1),
                                vals[b].double().repeat_interleave(QH // KVH, 1))
            tol = (2.0 ** -11 + 2.0 ** -18) * 5.5 + 2.0 ** -11 * want.abs()
            assert torch.all((out.double().cpu()[rows] - want).abs() <= tol), (new, b)
            wl = s.logsumexp(-1)
            assert torch.all((lse.double().cpu()[rows] - wl).abs() <= 1e-4 * wl.abs().clamp(min=1))
    # more tokens are cached than the pool has room for
    assert sum(len(x) for x in keys) > 100 and pool * P == 144
    assert sum(-(-len(x) // P) for x in keys) + st.count > pool
