"""GPU tests of attention with a sliding window and first tokens (single tokens,
and packed prompts and chunks) against a plain 64-bit statement.  Rows that no
query sees hold NaN, and pages without a visible row have wrong table entries."""
import math

import numpy as np
import pytest
import torch

import prompt_ref as ref
import window_ref as wref
from gpu_util import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _ok(fda, ws):
    st, info = fda.fd_check_device_error(ws)
    assert st == fda.FD_OK, (fda.fd_status_string(st), info)


def _queries(bt, qh, x16, seed):
    q = torch.randn((bt.tokens, qh, bt.d), generator=torch.Generator().manual_seed(seed))
    return q.to(ref.T16[x16])


def _decode(fda, f, q, window, sinks, ws, scale=None, **more):
    bt = f.batch
    kw = f.device(DEV)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    fda.decode_attention(q.to(DEV), kw.pop("k_cache"), kw.pop("v_cache"),
                         torch.tensor(bt.seq, dtype=torch.int32, device=DEV), out=out, lse=lse,
                         workspace=ws, softmax_scale=scale, window=window, sinks=sinks, **kw,
                         **bt.index(DEV), **more)
    torch.cuda.synchronize()
    return out.double().cpu(), lse.double().cpu()


def _prefill(fda, f, q, window, sinks, ws, scale=None, **more):
    bt = f.batch
    kw = f.device(DEV)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    fda.prefill_attention(q.to(DEV), kw.pop("k_cache"), kw.pop("v_cache"),
                          torch.from_numpy(bt.q_start).to(DEV),
                          torch.tensor(bt.seq, dtype=torch.int32, device=DEV), out=out, lse=lse,
                          workspace=ws, softmax_scale=scale, window=window, sinks=sinks, **kw,
                          **bt.index(DEV), **more)
    torch.cuda.synchronize()
    return out.double().cpu(), lse.double().cpu()


# ---------------------------------------------------------------------------
# single tokens
# ---------------------------------------------------------------------------

DECODE = [
    # lengths, qh, kvh, d, x16, kv, page, scales, window, sinks
    ([1, 2, 700, 33], 8, 2, 64, "bf16", "bf16", 0, "tensor", 64, 4),
    ([500, 1000, 3], 64, 8, 128, "f16", "e4m3", 64, "tensor", 100, 4),
    ([500, 1000, 3], 64, 8, 128, "f16", "e4m3", 16, "tensor", 100, 33),
    ([900, 40, 2000], 16, 1, 128, "bf16", "i8", 0, "token", 513, 64),
    ([900, 40, 2000], 16, 1, 128, "f16", "i8", 16, "token", 300, 3),
    ([0, 1, 300], 4, 4, 128, "f16", "f16", 1, "tensor", 1, 0),
    ([5000, 257], 128, 1, 128, "f16", "e4m3", 64, "tensor", 1024, 1),
    ([5000, 257], 96, 1, 64, "bf16", "i8", 8, "head", 999, 130),
    ([600, 601, 602], 12, 3, 64, "f16", "i8", 256, "token", 7, 1),
    ([600, 601, 602], 8, 8, 128, "f16", "i8", 256, "tensor", 255, 300),
    ([129, 640], 8, 8, 128, "bf16", "bf16", 64, "tensor", 130, 0),
    ([129, 640], 40, 2, 128, "f16", "f16", 4, "tensor", 131, 5),
    ([3000, 64], 24, 2, 128, "bf16", "e4m3", 2, "token", 640, 40),
    ([100, 64], 8, 2, 128, "bf16", "e4m3", 0, "head", 1 << 30, 0),
    ([100, 64], 8, 2, 128, "bf16", "e4m3", 0, "head", 16, (1 << 31) - 1),
]


@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode(case):
    fda = lib()
    lens, qh, kvh, d, x16, kv, page, scales, window, sinks = DECODE[case]
    bt = ref.Batch([1] * len(lens), [x - 1 for x in lens], kvh, d, kv, page, seed=case)
    f = ref.Filled(bt, scales, seed=case)
    wref.hide(f, window, sinks)
    q = _queries(bt, qh, x16, case)
    ws = fda.alloc_workspace(len(lens), qh, kvh, d)
    out, lse = _decode(fda, f, q, window, sinks, ws)
    _ok(fda, ws)
    want, wlse = wref.attention(f, q, qh, d ** -0.5, window, sinks)
    wref.compare(bt, out, lse, want, wlse, x16, str(DECODE[case]))


@pytest.mark.parametrize("seed", range(24))
def test_decode_many_sequences(seed):
    """Random batches: every format, layout and head grouping, windows and first
    tokens of all sizes, so that CTAs pass many streams, whole and cut, with and
    without a hidden middle."""
    fda = lib()
    rng = np.random.default_rng(500 + seed)
    kvh, group = [(8, 8), (2, 8), (1, 16), (4, 3), (8, 1), (3, 5), (1, 64), (2, 40)][seed % 8]
    d = 64 if seed % 3 == 0 else 128
    x16 = ["f16", "bf16"][seed % 2]
    kv = [x16, "e4m3", "i8"][(seed // 2) % 3]
    scales = ["tensor", "head", "token"][(seed // 6) % 3] if kv in ref.QMAX else "tensor"
    page = [0, 16, 64, 4, 256, 8, 1, 128][(seed // 3) % 8]
    window = int(rng.choice([1, 5, 31, 64, 100, 256, 257, 700]))
    sinks = int(rng.choice([0, 0, 1, 4, 32, 33, 300]))
    B = int(rng.integers(20, 70))
    lens = [int(x) for x in rng.choice([0, 1, 2, 31, 64, 100, 255, 256, 300, 513, 900, 1500], B)]
    bt = ref.Batch([1] * B, [x - 1 for x in lens], kvh, d, kv, page, seed=seed)
    f = ref.Filled(bt, scales, seed=seed)
    wref.hide(f, window, sinks)
    q = _queries(bt, kvh * group, x16, seed)
    ws = fda.alloc_workspace(B, kvh * group, kvh, d)
    out, lse = _decode(fda, f, q, window, sinks, ws)
    _ok(fda, ws)
    want, wlse = wref.attention(f, q, kvh * group, d ** -0.5, window, sinks)
    wref.compare(bt, out, lse, want, wlse, x16,
                 f"{kvh}x{group} d{d} {x16}/{kv} {scales} page {page} W {window} S {sinks}")
    again, lagain = _decode(fda, f, q, window, sinks, ws)
    assert torch.equal(out, again) and torch.equal(lse, lagain)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 2.0])
@pytest.mark.parametrize("kv,scales", [("f16", "tensor"), ("e4m3", "token"), ("i8", "head")])
def test_score_scales(scale, kv, scales):
    fda = lib()
    bt = ref.Batch([1, 1, 1], [69, 800, 900], 2, 128, kv, 16, seed=5)
    f = ref.Filled(bt, scales, seed=5)
    wref.hide(f, 200, 7)
    q = _queries(bt, 8, "f16", 5)
    want, wlse = wref.attention(f, q, 8, scale, 200, 7)
    ws = fda.alloc_workspace(3, 8, 2, 128)
    wref.compare(bt, *_decode(fda, f, q, 200, 7, ws, scale=scale), want, wlse, "f16")
    _ok(fda, ws)
    ws = fda.alloc_prefill_workspace(128)
    wref.compare(bt, *_prefill(fda, f, q, 200, 7, ws, scale=scale), want, wlse, "f16")
    _ok(fda, ws)


def test_a_window_longer_than_the_sequences_changes_nothing():
    """The same plan and the same arithmetic as without one: the same bits."""
    fda = lib()
    bt = ref.Batch([1, 1, 1, 1], [0, 299, 4000, 63], 2, 128, "e4m3", 16, seed=2)
    f = ref.Filled(bt, seed=2)
    q = _queries(bt, 16, "f16", 2)
    ws = fda.alloc_workspace(4, 16, 2, 128)
    for window, sinks in ((4001, 0), ((1 << 31) - 1, 9), (1, 4001)):
        a = _decode(fda, f, q, window, sinks, ws)
        b = _decode(fda, f, q, None, 0, ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    bt = ref.Batch([300, 1, 40, 7], [0, 2000, 260, -2], 2, 128, "bf16", 0, seed=2)
    f = ref.Filled(bt, seed=2)
    q = _queries(bt, 8, "bf16", 2)
    ws = fda.alloc_prefill_workspace(128)
    for window, sinks in ((2001, 0), ((1 << 31) - 1, 9), (1, 2001)):
        a = _prefill(fda, f, q, window, sinks, ws)
        b = _prefill(fda, f, q, None, 0, ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_with_its_append():
    """The step's new token is written first; with a window of one it is all
    that the query sees besides the first tokens."""
    fda = lib()
    for window, sinks in ((1, 0), (1, 2), (50, 0)):
        bt = ref.Batch([1] * 4, [0, 1, 70, 300], 2, 128, "i8", 16, seed=3)
        f = ref.Filled(bt, "token", seed=3)
        wref.hide(f, window, sinks)
        g = torch.Generator().manual_seed(4)
        kn, vn = (torch.randn((4, 2, 128), generator=g).half() for _ in range(2))
        rows = torch.tensor([bt.row(b, c) for b, c in enumerate(bt.ctx)])
        for w, x in (("k", kn), ("v", vn)):
            codes, tok = ref.quantise(x.float(), "i8", f.kw[w + "_scale"], None, "token")
            f.val[w][rows] = ref.value_of(codes, "i8") * (f.kw[w + "_scale"] * tok.double())[..., None]
        q = _queries(bt, 8, "f16", 3)
        ws = fda.alloc_workspace(4, 8, 2, 128)
        out, lse = _decode(fda, f, q, window, sinks, ws, k_new=kn.to(DEV), v_new=vn.to(DEV),
                           positions=torch.tensor(bt.ctx, dtype=torch.int32, device=DEV))
        _ok(fda, ws)
        want, wlse = wref.attention(f, q, 8, 128 ** -0.5, window, sinks)
        wref.compare(bt, out, lse, want, wlse, "f16")


def test_decode_rows_outside_the_cache():
    """A visible page outside the cache is recorded, a hidden one is not."""
    fda = lib()
    bt = ref.Batch([1], [299], 2, 128, "f16", 16, seed=1)
    f = ref.Filled(bt, seed=1)
    q = _queries(bt, 16, "f16", 1)
    ws = fda.alloc_workspace(1, 16, 2, 128)
    bt.block_table[0, 3] = 10 ** 6
    _decode(fda, f, q, 100, 4, ws)
    _ok(fda, ws)
    bt.block_table[0, 17] = 10 ** 6
    _decode(fda, f, q, 100, 4, ws)
    assert fda.fd_check_device_error(ws) == (fda.FD_ERR_DEVICE_BOUNDS, 10 ** 6)
    bt.block_table[0, 17] = 0
    wsp = fda.alloc_prefill_workspace(128)
    _prefill(fda, f, q, 100, 4, wsp)
    _ok(fda, wsp)
    bt.block_table[0, 0] = -7
    _prefill(fda, f, q, 100, 4, wsp)
    assert fda.fd_check_device_error(wsp) == (fda.FD_ERR_DEVICE_BOUNDS, -7)


def test_decode_sequences_longer_than_their_row_of_the_table():
    """What lies past the row's end is absent and recorded, the first tokens are
    seen; the next sequence's entries, which follow in memory, are not read."""
    fda = lib()
    for page, d in ((16, 128), (2, 64), (64, 128)):
        bt = ref.Batch([1, 1], [8 * page - 1, 5], 2, d, "f16", page, seed=1)
        f = ref.Filled(bt, seed=1)
        q = _queries(bt, 16, "f16", 1)
        want, wlse = wref.attention(f, q, 16, d ** -0.5, 7, 3)
        ws = fda.alloc_workspace(2, 16, 2, d)
        kw = f.device(DEV)
        args = (q.to(DEV), kw.pop("k_cache"), kw.pop("v_cache"))
        out, lse = fda.decode_attention(
            *args, torch.tensor([4000 * page, 6], dtype=torch.int32, device=DEV), window=7, sinks=3,
            workspace=ws, **kw, **bt.index(DEV))
        torch.cuda.synchronize()
        assert fda.fd_check_device_error(ws)[0] == fda.FD_ERR_DEVICE_BOUNDS
        s = torch.einsum("hd,khd->hk", q[0].double(),
                         f.val["k"][bt.rows_of(0, 0, 3)].repeat_interleave(8, 1)) / d ** 0.5
        only = torch.einsum("hk,khd->hd", s.softmax(-1),
                            f.val["v"][bt.rows_of(0, 0, 3)].repeat_interleave(8, 1))
        tol = (2.0 ** -11 + 2.0 ** -18) * 5.5 + 2.0 ** -11 * only.abs()
        assert torch.all((out[0].double().cpu() - only).abs() <= tol)
        tol = (2.0 ** -11 + 2.0 ** -18) * 5.5 + 2.0 ** -11 * want[1].abs()
        assert torch.all((out[1].double().cpu() - want[1]).abs() <= tol)


def test_forced_kernels():
    fda = lib()
    bt = ref.Batch([1, 1], [80, 300], 2, 128, "e4m3", 0, seed=1)
    f = ref.Filled(bt, seed=1)
    q = _queries(bt, 64, "f16", 1)
    ws = fda.alloc_workspace(2, 64, 2, 128)
    want = _decode(fda, f, q, 60, 4, ws)
    try:
        fda.fd_set_kernel(fda.FD_KERNEL_MMA)
        got = _decode(fda, f, q, 60, 4, ws)
        assert torch.equal(got[0], want[0])
        for k in (fda.FD_KERNEL_SIMT, fda.FD_KERNEL_TC, fda.FD_KERNEL_FMA):
            fda.fd_set_kernel(k)
            with pytest.raises(fda.FdError) as e:
                _decode(fda, f, q, 60, 4, ws)
            assert e.value.status == fda.FD_ERR_UNSUPPORTED
    finally:
        fda.fd_set_kernel(fda.FD_KERNEL_AUTO)


# ---------------------------------------------------------------------------
# packed prompts and chunks
# ---------------------------------------------------------------------------

PREFILL = [
    # new, ctx, qh, kvh, d, x16, kv, page, scales, window, sinks
    ([7, 333], [0, 0], 4, 1, 64, "f16", "f16", 0, "tensor", 65, 1),
    ([1, 1, 1], [0, 127, 700], 8, 2, 128, "bf16", "bf16", 16, "tensor", 128, 4),
    ([130, 0, 5], [0, 9, 700], 8, 2, 128, "f16", "f16", 64, "tensor", 100, 0),
    ([300], [0], 2, 2, 128, "bf16", "bf16", 0, "tensor", 1, 0),
    ([257, 64], [100, 1000], 6, 2, 64, "bf16", "bf16", 8, "tensor", 77, 9),
    ([40, 3], [733, 0], 10, 2, 128, "f16", "f16", 1, "tensor", 200, 129),
    ([9, 128], [4, 860], 5, 1, 64, "f16", "f16", 4, "tensor", 16, 3),
    ([128, 129], [0, 983], 16, 2, 128, "f16", "e4m3", 64, "tensor", 300, 16),
    ([61, 2], [1000, 255], 8, 8, 128, "bf16", "e4m3", 0, "head", 129, 130),
    ([100, 1], [529, 2000], 4, 1, 64, "f16", "e4m3", 16, "token", 333, 5),
    ([77, 1], [0, 515], 8, 1, 128, "f16", "i8", 16, "tensor", 40, 0),
    ([50, 50], [700, 250], 32, 8, 128, "bf16", "i8", 256, "token", 128, 2),
    ([19, 200], [0, 505], 12, 12, 64, "bf16", "i8", 2, "head", 255, 31),
    ([4, 1], [3000, 5000], 128, 1, 128, "f16", "e4m3", 64, "tensor", 1024, 4),
    ([6, 1], [700, 20], 65, 1, 128, "f16", "i8", 8, "token", 3, 100),
    ([500], [900], 1, 1, 128, "bf16", "i8", 16, "token", 256, 16),
    ([500, 20], [900, 5], 4, 4, 128, "f16", "f16", 0, "tensor", 127, 257),
    ([200, 3, 5, 40], [-190, -3, -2, 400], 4, 2, 64, "bf16", "bf16", 16, "tensor", 6, 2),
    ([70, 9], [700, 0], 4, 2, 64, "f16", "i8", 0, "token", (1 << 31) - 1, 0),
    ([70, 9], [700, -4], 4, 2, 64, "f16", "i8", 0, "token", 20, (1 << 31) - 1),
]


@pytest.mark.parametrize("case", range(len(PREFILL)))
def test_prefill(case):
    fda = lib()
    new, ctx, qh, kvh, d, x16, kv, page, scales, window, sinks = PREFILL[case]
    bt = ref.Batch(new, ctx, kvh, d, kv, page, seed=case, lead=2, tail=3)
    f = ref.Filled(bt, scales, seed=case)
    wref.hide(f, window, sinks)
    q = _queries(bt, qh, x16, case)
    ws = fda.alloc_prefill_workspace(d)
    out, lse = _prefill(fda, f, q, window, sinks, ws)
    _ok(fda, ws)
    want, wlse = wref.attention(f, q, qh, d ** -0.5, window, sinks)
    wref.compare(bt, out, lse, want, wlse, x16, str(PREFILL[case]))


@pytest.mark.parametrize("seed", range(24))
def test_prefill_many_streams(seed):
    fda = lib()
    rng = np.random.default_rng(700 + seed)
    kvh, group = [(8, 1), (2, 8), (1, 16), (4, 3), (8, 4), (3, 5)][seed % 6]
    d = 64 if seed % 4 else 128
    x16 = ["f16", "bf16"][seed % 2]
    kv = [x16, "e4m3", "i8"][(seed // 2) % 3]
    scales = ["tensor", "head", "token"][(seed // 6) % 3] if kv in ref.QMAX else "tensor"
    page = [0, 16, 64, 4, 256, 8][(seed // 3) % 6]
    window = int(rng.choice([1, 5, 64, 100, 128, 129, 300]))
    sinks = int(rng.choice([0, 0, 1, 4, 128, 150]))
    B = int(rng.integers(30, 70))
    new = [int(x) for x in rng.choice([0, 1, 1, 2, 17, 40, 90], B)]
    ctx = [int(x) for x in rng.choice([0, 0, 1, 100, 127, 128, 300, 600, -1], B)]
    new[0], ctx[0] = 300, 340
    ctx = [max(c, -n) for n, c in zip(new, ctx)]
    bt = ref.Batch(new, ctx, kvh, d, kv, page, seed=seed, lead=1, tail=2)
    f = ref.Filled(bt, scales, seed=seed)
    wref.hide(f, window, sinks)
    q = _queries(bt, kvh * group, x16, seed)
    ws = fda.alloc_prefill_workspace(d)
    out, lse = _prefill(fda, f, q, window, sinks, ws)
    _ok(fda, ws)
    want, wlse = wref.attention(f, q, kvh * group, d ** -0.5, window, sinks)
    wref.compare(bt, out, lse, want, wlse, x16,
                 f"{kvh}x{group} d{d} {x16}/{kv} {scales} page {page} W {window} S {sinks}")
    again, lagain = _prefill(fda, f, q, window, sinks, ws)
    assert torch.equal(out, again) and torch.equal(lse, lagain)


def test_prefill_many_tokens():
    """Long prompts, so that streams are cut and merged with gaps in them."""
    fda = lib()
    for kv, page, x16, window, sinks in (("bf16", 0, "bf16", 1024, 0), ("e4m3", 64, "f16", 500, 4),
                                         ("i8", 16, "bf16", 1500, 200)):
        bt = ref.Batch([2500, 1, 700], [0, 3000, 1900], 1, 128, kv, page, seed=11)
        f = ref.Filled(bt, "token" if kv == "i8" else "tensor", seed=11)
        wref.hide(f, window, sinks)
        q = _queries(bt, 4, x16, 11)
        ws = fda.alloc_prefill_workspace(128)
        out, lse = _prefill(fda, f, q, window, sinks, ws)
        _ok(fda, ws)
        want, wlse = wref.attention(f, q, 4, 128 ** -0.5, window, sinks)
        wref.compare(bt, out, lse, want, wlse, x16, kv)


@pytest.mark.parametrize("kv,page,window,sinks", [("bf16", 0, 50, 3), ("f16", 16, 200, 0),
                                                  ("bf16", 4, 64, 10), ("e4m3", 16, 100, 140),
                                                  ("e4m3", 0, 33, 1), ("e4m3", 2, 128, 0)])
def test_prefill_nonfinite_values_stay_with_their_readers(kv, page, window, sinks):
    """NaN and infinite V elements reach the tokens that see them, on both ends
    of the window and among the first tokens, and no other."""
    fda = lib()
    x16 = kv if kv in ref.T16 else "f16"
    bt = ref.Batch([90, 300, 30], [20, 0, 400], 2, 64, kv, page, seed=7)
    f = ref.Filled(bt, seed=7)
    wref.hide(f, window, sinks)
    q = _queries(bt, 4, x16, 7)
    marks = [(0, 60, 0, 5, float("nan")), (1, 100, 1, 9, float("inf")), (1, 200, 1, 9, -math.inf),
             (1, 130, 0, 63, float("inf")), (2, 415, 1, 0, float("nan")), (1, 0, 0, 31, math.inf),
             (2, 380, 0, 7, float("inf")), (1, 128, 1, 40, float("nan"))]
    for b, t, h, dim, x in marks:
        row = bt.row(b, t)
        if kv == "e4m3":
            x = float("nan")
            f.kw["v_cache"].view(bt.rows, 2, 64)[row, h, dim] = 0x7F
        else:
            f.kw["v_cache"].view(bt.rows, 2, 64)[row, h, dim] = x
        f.val["v"][row, h, dim] = x
    ws = fda.alloc_prefill_workspace(64)
    out, lse = _prefill(fda, f, q, window, sinks, ws)
    _ok(fda, ws)
    want, wlse = wref.attention(f, q, 4, 64 ** -0.5, window, sinks)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(torch.isinf(out), torch.isinf(want))
    assert torch.equal(out[torch.isinf(out)], want[torch.isinf(want)])
    fin = torch.isfinite(want)
    eps = torch.finfo(ref.T16[x16]).eps
    assert torch.all((out - want)[fin].abs() <= (eps / 2 + 2.0 ** -18) * 5.5 + eps / 2 * want[fin].abs())
    assert float((lse - wlse).abs().max()) <= 1e-4 * max(1.0, float(wlse.abs().max()))


@pytest.mark.parametrize("x16", ["f16", "bf16"])
def test_prefill_scales_of_keys_that_leave_the_window(x16):
    """Per-token scales: a key's huge V scale costs only the tokens that see it,
    and a NaN one reaches only them."""
    fda = lib()
    bt = ref.Batch([150, 3], [300, 200], 1, 64, "i8", 16, seed=8)
    f = ref.Filled(bt, "token", seed=8)
    wref.hide(f, 100, 0)
    i = int(bt.q_start[0])
    row = bt.row(0, 240)     # seen by the tokens at 300 .. 339 only
    f.kw["v_scales"][row] *= 1e6
    f.val["v"][row] *= 1e6
    nan = bt.row(0, 230)     # seen by 300 .. 329
    f.kw["v_scales"][nan] = float("nan")
    f.val["v"][nan] = float("nan")
    q = _queries(bt, 4, x16, 8)
    ws = fda.alloc_prefill_workspace(64)
    out, lse = _prefill(fda, f, q, 100, 0, ws)
    _ok(fda, ws)
    want, wlse = wref.attention(f, q, 4, 64 ** -0.5, 100, 0)
    assert torch.isnan(out[i:i + 30]).all() and torch.isnan(want[i:i + 30]).all()
    far = slice(i + 40, bt.tokens)   # its own tolerance: nothing of the large scale is left
    eps = torch.finfo(ref.T16[x16]).eps
    tol = (eps / 2 + 2.0 ** -18) * 5.5 + eps / 2 * want[far].abs()
    assert torch.all((out[far] - want[far]).abs() <= tol)


# ---------------------------------------------------------------------------
# how programs call it
# ---------------------------------------------------------------------------

def test_window_steps_in_a_graph_and_on_other_streams():
    """A captured decode step and a captured chunk, replayed with new lengths,
    queries and table entries; and both on a stream of their own."""
    fda = lib()
    window, sinks = 70, 2
    for which in (_decode_call, _prefill_call):
        new = [1] * 3 if which is _decode_call else [30, 1, 8]
        a, b = ([40, 200, 500], [3, 499, 60])
        steps = [ref.Batch(new, x, 2, 128, "e4m3", 16, seed=i) for i, x in enumerate((a, b, a))]
        bt = steps[0]
        cols = max(x.block_table.shape[1] for x in steps)
        rows = max(x.rows for x in steps)
        table = torch.zeros((3, cols), dtype=torch.int32, device=DEV)
        kc, vc = (torch.zeros((rows // 16, 16, 2, 128), dtype=torch.uint8, device=DEV)
                  for _ in range(2))
        q = torch.zeros((sum(new), 16, 128), dtype=torch.float16, device=DEV)
        seq = torch.zeros(3, dtype=torch.int32, device=DEV)
        qs = torch.from_numpy(bt.q_start).to(DEV)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
        ws = which(fda, None, *[None] * 9, window, sinks, make=True)
        side = torch.cuda.Stream()
        graph = None
        for k, x in enumerate(steps):
            f = ref.Filled(x, seed=k)
            wref.hide(f, window, sinks)
            hq = _queries(x, 16, "f16", k)
            table.fill_(-1)
            table[:, :x.block_table.shape[1]] = torch.from_numpy(x.block_table).to(DEV)
            for c, w in ((kc, "k"), (vc, "v")):
                c.view(rows, 2, 128)[:x.rows] = f.kw[w + "_cache"].view(x.rows, 2, 128).to(DEV)
            q.copy_(hq)
            seq.copy_(torch.tensor(x.seq, dtype=torch.int32))
            out.fill_(7.0)
            scale = f.kw["k_scale"]
            torch.cuda.synchronize()
            args = (q, kc, vc, seq, qs, table, scale, out, lse, window, sinks)
            if graph is None:
                with torch.cuda.stream(side):   # another stream first
                    which(fda, ws, *args, stream=side)
                side.synchronize()
                _check(x, f, hq, out, lse, window, sinks)
                out.fill_(7.0)
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    which(fda, ws, *args)
            graph.replay()
            torch.cuda.synchronize()
            _ok(fda, ws)
            _check(x, f, hq, out, lse, window, sinks)


def _check(bt, f, q, out, lse, window, sinks):
    want, wlse = wref.attention(f, q, 16, 128 ** -0.5, window, sinks)
    wref.compare(bt, out.double().cpu(), lse.double().cpu(), want, wlse, "f16")


def _decode_call(fda, ws, q, kc, vc, seq, qs, table, scale, out, lse, window, sinks, make=False,
                 **kw):
    if make:
        return fda.alloc_workspace(3, 16, 2, 128)
    fda.decode_attention(q, kc, vc, seq, block_table=table, k_scale=scale, v_scale=scale,
                         workspace=ws, out=out, lse=lse, window=window, sinks=sinks, **kw)


def _prefill_call(fda, ws, q, kc, vc, seq, qs, table, scale, out, lse, window, sinks, make=False,
                  **kw):
    if make:
        return fda.alloc_prefill_workspace(128)
    fda.prefill_attention(q, kc, vc, qs, seq, block_table=table, k_scale=scale, v_scale=scale,
                          workspace=ws, out=out, lse=lse, window=window, sinks=sinks, **kw)


def test_window_waits_that_run_out_are_reported():
    """With a producer that issues no copy, the waits give up after their limit
    and the call is reported as a timeout; the next call works."""
    fda = lib()
    bt = ref.Batch([1, 1], [300, 900], 8, 128, "e4m3", 0, seed=1)
    f = ref.Filled(bt, seed=1)
    q = _queries(bt, 64, "f16", 1)
    ws, wsp = fda.alloc_workspace(2, 64, 8, 128), fda.alloc_prefill_workspace(128)
    try:
        fda.fd_debug_set_wait_limit(2000000, True)
        _decode(fda, f, q, 100, 4, ws)
        assert fda.fd_check_device_error(ws)[0] == fda.FD_ERR_DEVICE_TIMEOUT
        _prefill(fda, f, q, 100, 4, wsp)
        assert fda.fd_check_device_error(wsp)[0] == fda.FD_ERR_DEVICE_TIMEOUT
    finally:
        fda.fd_debug_set_wait_limit(0, False)
    want, wlse = wref.attention(f, q, 64, 128 ** -0.5, 100, 4)
    wref.compare(bt, *_decode(fda, f, q, 100, 4, ws), want, wlse, "f16")
    wref.compare(bt, *_prefill(fda, f, q, 100, 4, wsp), want, wlse, "f16")
    _ok(fda, ws)
    _ok(fda, wsp)


def test_window_far_into_a_large_cache():
    """Rows whose byte offsets pass 32 bits, at both ends of the window's gap."""
    fda = lib()
    rows, d = 40_000_000, 128
    kc, vc = (torch.zeros((rows, 1, d), dtype=torch.uint8, device=DEV) for _ in range(2))
    T, window, sinks = 36_000_000, 300, 5
    start = rows - T
    g = torch.Generator().manual_seed(1)
    seen = [t for t in range(sinks)] + [t for t in range(T - window - 9, T)]
    k, v = (torch.randn((len(seen), d), generator=g).to(torch.float8_e4m3fn) for _ in range(2))
    at = torch.tensor(seen, device=DEV) + start
    kc[at, 0] = k.view(torch.uint8).to(DEV)
    vc[at, 0] = v.view(torch.uint8).to(DEV)
    q = torch.randn((10, 8, d), generator=g).half()
    kv = dict(kv_start_idx=torch.tensor([start], dtype=torch.int32, device=DEV))
    seq = torch.tensor([T], dtype=torch.int32, device=DEV)
    qs = torch.tensor([0, 10], dtype=torch.int32, device=DEV)
    out, lse = fda.prefill_attention(q.to(DEV), kc, vc, qs, seq, window=window, sinks=sinks, **kv)
    one, l1 = fda.decode_attention(q[9:].to(DEV), kc, vc, seq, window=window, sinks=sinks, **kv)
    torch.cuda.synchronize()
    t = torch.tensor(seen)[None, :]
    p = (T - 10 + torch.arange(10))[:, None]
    ok = (t <= p) & ((t > p - window) | (t < sinks))
    s = torch.einsum("qhd,kd->qhk", q.double(), k.double()) / d ** 0.5
    s = s.masked_fill(~ok[:, None, :], -math.inf)
    want = torch.einsum("qhk,kd->qhd", s.softmax(-1), v.double())
    eps = 2.0 ** -10
    tol = (eps / 2 + 2.0 ** -18) * 5.5 + eps / 2 * want.abs()
    assert torch.all((out.double().cpu() - want).abs() <= tol)
    assert torch.all((one.double().cpu() - want[9:]).abs() <= tol[9:])
    wl = s.logsumexp(-1)
    assert float((lse.double().cpu() - wl).abs().max()) <= 1e-4 * float(wl.abs().max())
    assert float((l1.double().cpu() - wl[9:]).abs().max()) <= 1e-4 * float(wl.abs().max())
