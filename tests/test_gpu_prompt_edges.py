"""GPU tests of the prompt path at its edges: finite and non-finite scales and
values in places a row may not see, absent tiles, empty calls, wrong starts,
refusals that leave the caches alone, waits that run out in the middle."""
import math

import numpy as np
import pytest
import torch

import prompt_ref as ref
from gpu_util import lib
from test_gpu_prompt import DEV, _attend, _compare, _ok, _queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x16", ["f16", "bf16"])
@pytest.mark.parametrize("kv,page,d", [("i8", 16, 64), ("e4m3", 0, 128), ("i8", 2, 128)])
def test_attention_scales_of_unseen_keys_have_no_effect(kv, page, d, x16):
    """However large the K and V scales of a token are, the tokens before it get
    the same bits; and each row is right against the keys that it sees."""
    fda = lib()
    bt = ref.Batch([100, 40, 200, 1], [0, 300, 70, 500], 2, d, kv, page, seed=31)
    f = ref.Filled(bt, "token", seed=31)
    q = _queries(bt, 8, x16, 31)
    ws = fda.alloc_prefill_workspace(d)
    base, lbase = _attend(fda, f, q, 8, ws)
    late = {b: int(bt.seq[b] - min(17, bt.new[b])) for b in range(len(bt.new))}   # first large one
    for big in (2.0 ** 20, 1e12, 3e38):
        for b, T in enumerate(bt.seq):
            rows = bt.rows_of(b, late[b], T)
            f.kw["v_scales"][rows] = big
            f.kw["k_scales"][rows] = big
        out, lse = _attend(fda, f, q, 8, ws)
        _ok(fda, ws)
        for b, n in enumerate(bt.new):
            i = int(bt.q_start[b])
            m = n - (bt.seq[b] - late[b])     # rows that see none of them
            assert torch.equal(out[i:i + m], base[i:i + m]), (big, b)
            assert torch.equal(lse[i:i + m], lbase[i:i + m]), (big, b)


def test_attention_value_scales_row_by_row():
    """V scales that grow along the sequence, f16 queries: each row against the
    largest value that it sees itself."""
    fda = lib()
    bt = ref.Batch([128, 300, 7], [0, 100, 600], 2, 64, "i8", 16, seed=32)
    f = ref.Filled(bt, "token", seed=32)
    old = f.kw["v_scales"].clone()
    for b, T in enumerate(bt.seq):
        rows = bt.rows_of(b, 0, T)
        grow = 2.0 ** (torch.arange(T, dtype=torch.float64) * (28.0 / T) - 16)
        f.kw["v_scales"][rows] = (old[rows].double() * grow[:, None]).float()
    ratio = f.kw["v_scales"].double() / old.double()
    f.val["v"] = f.val["v"] * ratio[:, :, None]
    q = _queries(bt, 4, "f16", 32)
    ws = fda.alloc_prefill_workspace(64)
    out, lse = _attend(fda, f, q, 4, ws)
    _ok(fda, ws)
    want, wlse = ref.attention_blocks(f, q, 4, 0.125)
    assert float((lse - wlse).abs().max()) <= 1e-4
    # sum p |v| of every row, and the largest |v| that it sees
    mag = ref.Filled(bt, "token", seed=32)
    mag.val["v"] = f.val["v"].abs()
    weight, _ = ref.attention_blocks(mag, q, 4, 0.125)
    top = torch.zeros(want.shape[:2], dtype=torch.float64)
    seen = torch.zeros(want.shape[0], dtype=torch.float64)
    for b, n in enumerate(bt.new):
        for j in range(n):
            i, t = int(bt.q_start[b]) + j, bt.seq[b] - n + j + 1
            seen[i] = t
            if j == 0:
                run = f.val["v"][bt.rows_of(b, 0, t)].abs().amax(dim=(0, 2))
            else:
                run = torch.maximum(run, f.val["v"][bt.row(b, t - 1)].abs().amax(-1))
            top[i] = run.repeat_interleave(2)
    # P times a V scale is rounded to f16: half a step, 2^-11 of itself, or
    # below f16's normal range 2^-25, with P lifted by 2^6 against the largest
    # scale seen: 2^-31 of that scale times the key's code, which is below eight
    # times the largest code of the key with that scale: 2^-28 of the largest
    # |v| for every key.  The output is rounded once more (2^-11, or half of its
    # own subnormal step); fp32 sums and ex2 2^-18.
    tol = ((2.0 ** -11 + 2.0 ** -18) * weight + (seen[:, None] * 2.0 ** -28 * top)[..., None] +
           2.0 ** -11 * want.abs() + 2.0 ** -25)
    assert torch.all((out - want).abs() <= tol), float(((out - want).abs() / tol).max())


def _absent_statement(f, q, qh, b, tile, scale):
    """Sequence b without the keys of one 128-key tile: [new, qh, d] in 64 bits."""
    bt = f.batch
    n, T, g = bt.new[b], bt.seq[b], qh // bt.kvh
    keys = torch.tensor([t for t in range(T) if t // 128 != tile])
    rows = torch.tensor([bt.row(b, int(t)) for t in keys])
    out = torch.zeros((n, qh, bt.d), dtype=torch.float64)
    for j in range(n):
        see = keys <= T - n + j
        if not bool(see.any()):
            continue
        for h in range(qh):
            s = q[int(bt.q_start[b]) + j, h].double() @ f.val["k"][rows[see], h // g].T * scale
            out[j, h] = torch.softmax(s, -1) @ f.val["v"][rows[see], h // g]
    return out


@pytest.mark.parametrize("x16", ["f16", "bf16"])
def test_attention_absent_tile_with_bad_scales(x16):
    """A tile with a row outside the cache is absent, whatever the scales of its
    other rows are."""
    fda = lib()
    bt = ref.Batch([30], [300], 1, 64, "i8", 16, seed=33)
    f = ref.Filled(bt, "token", seed=33)
    q = _queries(bt, 2, x16, 33)
    want = _absent_statement(f, q, 2, 0, 1, 0.125)
    for t, bad in ((130, float("nan")), (131, float("inf")), (132, 3e38)):
        f.kw["v_scales"][bt.row(0, t)] = bad
    good = bt.block_table.copy()
    bt.block_table[0, 10] = 10 ** 6                # keys 160 .. 175
    ws = fda.alloc_prefill_workspace(64)
    out, lse = _attend(fda, f, q, 2, ws)
    assert fda.fd_check_device_error(ws) == (fda.FD_ERR_DEVICE_BOUNDS, 10 ** 6)
    bt.block_table = good
    eps = torch.finfo(ref.T16[x16]).eps
    assert torch.all((out - want).abs() <= (eps / 2 + 2.0 ** -18) * 5.5 + eps / 2 * want.abs())


@pytest.mark.parametrize("kv,page", [("f16", 16), ("bf16", 4), ("e4m3", 16)])
def test_attention_absent_tile_with_bad_values(kv, page):
    """Non-finite V elements of an absent tile reach nobody, though the pair of
    query tiles repairs those of another tile."""
    fda = lib()
    x16 = kv if kv in ref.T16 else "f16"
    # streams enough that whole pairs of query tiles, two tiles each, stay in one
    # block's segment
    bt = ref.Batch([250] * 24, [0] * 24, 8, 64, kv, page, seed=34)
    f = ref.Filled(bt, seed=34)
    q = _queries(bt, 8, x16, 34)
    cache = f.kw["v_cache"].view(bt.rows, 8, 64)
    nan = 0x7F if kv == "e4m3" else float("nan")
    good = bt.block_table.copy()
    some = range(3, 24, 5)
    want = {}
    for b in some:
        cache[bt.row(b, 5), :, 9] = nan            # in the absent tile
        cache[bt.row(b, 200), :, 3] = nan
        f.val["v"][bt.row(b, 200), :, 3] = float("nan")
        want[b] = _absent_statement(f, q, 8, b, 0, 0.125)
        bt.block_table[b, 64 // page] = -9         # keys from 64 on
    ws = fda.alloc_prefill_workspace(64)
    out, lse = _attend(fda, f, q, 8, ws)
    assert fda.fd_check_device_error(ws) == (fda.FD_ERR_DEVICE_BOUNDS, -9)
    bt.block_table = good
    eps = torch.finfo(ref.T16[x16]).eps
    for b in some:
        o, w = out[int(bt.q_start[b]):int(bt.q_start[b + 1])], want[b]
        assert torch.equal(torch.isnan(o), torch.isnan(w)), b
        fin = torch.isfinite(w)
        assert torch.all((o - w)[fin].abs() <=
                         (eps / 2 + 2.0 ** -18) * 5.5 + eps / 2 * w[fin].abs())


@pytest.mark.parametrize("kv,scales", [("f16", "tensor"), ("bf16", "tensor"), ("i8", "token")])
def test_attention_infinite_values_under_a_negative_scale(kv, scales):
    """v_scale times an infinite V element: the sign is that of the product, in
    streams of one block and in cut ones."""
    fda = lib()
    x16 = kv if kv in ref.T16 else "bf16"
    bt = ref.Batch([90, 300], [0, 2000], 2, 64, kv, 16, seed=35)
    f = ref.Filled(bt, scales, seed=35)
    q = _queries(bt, 4, x16, 35)
    for b, t, h, x in ((0, 40, 0, math.inf), (0, 60, 1, -math.inf), (1, 2100, 0, math.inf),
                       (1, 2290, 1, -math.inf)):
        row = bt.row(b, t)
        if scales == "token":      # every element of the row: by its code's sign
            f.kw["v_scales"][row, h] = x
            f.val["v"][row, h] = f.val["v"][row, h].sign() * x
        else:
            f.kw["v_cache"].view(bt.rows, 2, 64)[row, h, 7] = x
            f.val["v"][row, h, 7] = x
    if scales == "token":
        f.val["v"] = torch.where(torch.isnan(f.val["v"]), 1.0, f.val["v"])
    f.kw["v_scale"] = -0.5 * f.kw["v_scale"]
    f.val["v"] = -0.5 * f.val["v"]
    ws = fda.alloc_prefill_workspace(64)
    out, lse = _attend(fda, f, q, 4, ws)
    _ok(fda, ws)
    want, wlse = ref.attention(f, q, 4, 0.125)
    inf = torch.isinf(want)
    assert int(inf.sum()) > 0 and torch.equal(out[inf], want[inf])
    fin = torch.isfinite(want) & torch.isfinite(out)
    if scales != "token":      # (there 0 * inf is NaN where a code is zero)
        assert torch.equal(torch.isfinite(out), torch.isfinite(want))
    eps = torch.finfo(ref.T16[x16]).eps
    assert torch.all((out - want)[fin].abs() <=
                     (eps / 2 + 2.0 ** -18) * 5.5 * 0.5 + eps / 2 * want[fin].abs())


def test_calls_of_nothing():
    """No packed tokens, no rows: empty results, nothing written."""
    fda = lib()
    k = torch.full((8, 2, 64), 3.0, dtype=torch.float16, device=DEV)
    v = k.clone()
    i32 = dict(dtype=torch.int32, device=DEV)
    start, zero = torch.zeros(3, **i32), torch.zeros(2, **i32)
    for base in (torch.empty((0, 4, 64), dtype=torch.float16, device=DEV),
                 torch.ones((9, 4, 64), dtype=torch.float16, device=DEV)[4:4]):
        new = base[:, :2]
        q = fda.append_kv(new, new, k, v, start, zero, q=base, kv_start_idx=zero)
        assert tuple(q.shape) == (0, 4, 64)
        assert fda.append_kv(new, new, k, v, start, zero, kv_start_idx=zero) is None
        out, lse = fda.prefill_attention(base, k, v, start, zero, kv_start_idx=zero)
        assert tuple(out.shape) == (0, 4, 64) and tuple(lse.shape) == (0, 4)
        out, lse = fda.prefill_attention(base, k, v, start, zero, kv_start_idx=zero, k_new=new,
                                         v_new=new, positions=zero,
                                         rotary=fda.rotary_table(4, 64))
        assert tuple(out.shape) == (0, 4, 64) and tuple(lse.shape) == (0, 4)
    ko, vo = fda.read_kv(k, v, start, 0, kv_start_idx=zero)
    assert tuple(ko.shape) == tuple(vo.shape) == (0, 2, 64)
    torch.cuda.synchronize()
    assert bool((k == 3).all()) and bool((v == 3).all())


@pytest.mark.parametrize("starts,served", [
    ([0, -5, 50], []), ([0, 60, 50], []), ([30, 20, 50], [1]), ([0, 50, 60], [0]),
    ([0, 20, 70], [0]), ([0, 20, 20, 10, 50], [0])])
def test_wrong_starts_are_recorded(starts, served):
    """Starts that descend or lie outside the packed arrays: recorded by every
    packed call; rows behind the last start and before the first stay."""
    fda = lib()
    n, d, B = 50, 64, len(starts) - 1
    i32 = dict(dtype=torch.int32, device=DEV)
    qs = torch.tensor(starts, **i32)
    first = torch.arange(B, **i32) * 100
    pos = torch.zeros(B, **i32)
    new = torch.ones((n, 1, d), dtype=torch.float16, device=DEV)
    kc, vc = (torch.zeros((100 * B, 1, d), dtype=torch.float16, device=DEV) for _ in range(2))
    q_out = torch.zeros((n, 2, d), dtype=torch.float16, device=DEV)
    ws = fda.alloc_prefill_workspace(d)
    fda.append_kv(new, new, kc, vc, qs, pos, q=new.expand(n, 2, d).contiguous(), q_out=q_out,
                  kv_start_idx=first, workspace=ws)
    st, info = fda.fd_check_device_error(ws)
    assert st == fda.FD_ERR_DEVICE_BOUNDS and info in starts
    rows = kc[:, 0, 0].view(B, 100).sum(1).tolist()
    for b in served:
        lo = max(starts[b], starts[0])
        assert rows[b] == starts[b + 1] - lo, rows
    assert bool((q_out[starts[-1]:] == 0).all()) and bool((q_out[:starts[0]] == 0).all())
    ko, vo = (torch.full((n, 1, d), 9.0, dtype=torch.float16, device=DEV) for _ in range(2))
    fda.read_kv(kc, vc, qs, n, kv_start_idx=first, k_out=ko, v_out=vo, workspace=ws)
    st, info = fda.fd_check_device_error(ws)
    assert st == fda.FD_ERR_DEVICE_BOUNDS and info in starts
    assert bool((ko[starts[-1]:] == 9).all()) and bool((ko[:starts[0]] == 9).all())
    fda.prefill_attention(torch.ones((n, 2, d), dtype=torch.float16, device=DEV), kc, vc, qs,
                          torch.full((B,), 40, **i32), kv_start_idx=first, workspace=ws)
    st, info = fda.fd_check_device_error(ws)
    assert st == fda.FD_ERR_DEVICE_BOUNDS and info in starts


def test_refused_prompt_calls_write_nothing():
    """prefill_attention with new keys: every refusal comes before the caches
    are written."""
    fda = lib()
    i32 = dict(dtype=torch.int32, device=DEV)
    kc, vc = (torch.zeros((40, 2, 64), dtype=torch.float16, device=DEV) for _ in range(2))
    q = torch.ones((6, 4, 64), dtype=torch.float16, device=DEV)
    new = torch.ones((6, 2, 64), dtype=torch.float16, device=DEV)
    at = dict(kv_start_idx=torch.zeros(1, **i32), positions=torch.zeros(1, **i32))
    starts, lens = torch.tensor([0, 6], **i32), torch.tensor([6], **i32)

    def call(q=q, k_new=new, v_new=new, **kw):
        return fda.prefill_attention(q, kc, vc, starts, lens, k_new=k_new, v_new=v_new, **at, **kw)

    for error, kw in (
            (ValueError, dict(k_new=new[:5], v_new=new[:5])),       # fewer keys than queries
            (ValueError, dict(k_new=new[:5], v_new=new[:5], rotary=fda.rotary_table(8, 64))),
            (fda.FdError, dict(workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))),
            (fda.FdError, dict(softmax_scale=float("nan"))),
            ((ValueError, fda.FdError), dict(out=q))):               # read by other blocks
        with pytest.raises(error):
            call(**kw)
    torch.cuda.synchronize()
    assert int(kc.count_nonzero()) == 0 and int(vc.count_nonzero()) == 0
    # with a table the queries are turned into a tensor of the call's own
    mine = q.clone()
    out, lse = call(q=mine, out=mine, rotary=fda.rotary_table(8, 64))
    again, lagain = call(rotary=fda.rotary_table(8, 64))
    assert out is mine and torch.equal(out, again) and torch.equal(lse, lagain)


@pytest.mark.parametrize("kv,page,scales", [("f16", 0, "tensor"), ("bf16", 64, "tensor"),
                                            ("f16", 4, "tensor"), ("e4m3", 64, "tensor"),
                                            ("i8", 16, "token"), ("e4m3", 2, "token")])
def test_attention_waits_do_run_out(kv, page, scales):
    """With limits of a few tries of a barrier (a microsecond each), waits run
    out in a call at work: behind rows gathered one by one, and where the
    producer passes many empty sequences and then fills its ring for a block
    that has given up.  Every such call ends and says so, and the next one is
    right."""
    fda = lib()
    x16 = kv if kv in ref.T16 else "f16"
    none = [0] * (16000 if page in (0, 16, 64) else 0)
    bt = ref.Batch([300, 1] + none + [64, 3] + none + [1, 200],
                   [40, 3000] + none + [0, 900] + none + [5000, 1500], 4, 128, kv, page, seed=36)
    f = ref.Filled(bt, scales, seed=36)
    q = _queries(bt, 16, x16, 36)
    ws = fda.alloc_prefill_workspace(128)
    want, wlse = ref.attention_blocks(f, q, 16, 128 ** -0.5)
    junk = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    seen = []
    for limit in (1, 1000, 3000, 10000):
        fda.fd_debug_set_wait_limit(limit, False)
        try:
            for _ in range(4):
                junk.fill_(limit & 7)        # the caches' rows come from memory again
                _attend(fda, f, q, 16, ws)
                seen.append(fda.fd_check_device_error(ws)[0])
        finally:
            fda.fd_debug_set_wait_limit(0, False)
    print(kv, page, scales, seen)
    assert set(seen) <= {fda.FD_OK, fda.FD_ERR_DEVICE_TIMEOUT}
    assert fda.FD_ERR_DEVICE_TIMEOUT in seen[:4], seen
    out, lse = _attend(fda, f, q, 16, ws)
    _ok(fda, ws)
    _compare(f, out, lse, want, wlse, x16)


def test_attention_passes_millions_of_empty_sequences():
    """A batch of empty sequences with two prompts far apart: no wait for the
    warp that looks for the next prompt runs out."""
    fda = lib()
    B = 12 * 10 ** 6
    bt = ref.Batch([70, 50], [0, 0], 2, 64, "f16", 0, seed=37)
    f = ref.Filled(bt, seed=37)
    q = _queries(bt, 4, "f16", 37)
    kw = f.device(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    starts, lens, first = torch.full((B + 1,), 70, **i32), torch.zeros(B, **i32), torch.zeros(B, **i32)
    starts[0], starts[B] = 0, 120
    lens[0], lens[B - 1] = 70, 50
    first[0], first[B - 1] = int(bt.kv_start_idx[0]), int(bt.kv_start_idx[1])
    ws = fda.alloc_prefill_workspace(64)
    out, lse = fda.prefill_attention(q.to(DEV), kw["k_cache"], kw["v_cache"], starts, lens,
                                     kv_start_idx=first, workspace=ws)
    torch.cuda.synchronize()
    _ok(fda, ws)
    want, wlse = ref.attention_blocks(f, q, 4, 0.125)
    _compare(f, out.double().cpu(), lse.double().cpu(), want, wlse, "f16")
