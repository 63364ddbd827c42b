"""GPU tests of per-token scales behind a sliding window: pages that no query
sees, whose entries still name pages with NaN and infinite scales."""
import pytest
import torch

import prompt_ref as ref
import window_ref as wref
from gpu_util import lib
from test_gpu_window import DEV, _decode, _ok, _prefill, _queries

pytestmark = pytest.mark.gpu


def _hidden(bt, scales_of, window, sinks, seed):
    """Hidden rows and their scales are poison, their pages' entries stay."""
    f = ref.Filled(bt, "token", seed=seed)
    table = bt.block_table.copy()
    cut = wref.hide(f, window, sinks)
    assert cut > 0
    bt.block_table[:] = table
    for w in "kv":
        x = f.kw[w + "_scales"]
        x[torch.isnan(x)] = scales_of[w]
    return f


@pytest.mark.parametrize("scales_of", [dict(k=float("nan"), v=float("inf")),
                                       dict(k=float("-inf"), v=float("nan"))])
@pytest.mark.parametrize("kvh,page,x16,kv", [(1, 16, "bf16", "i8"), (2, 4, "f16", "i8"),
                                             (2, 64, "f16", "e4m3"), (8, 16, "bf16", "e4m3"),
                                             (3, 128, "f16", "i8")])
def test_scales_of_hidden_pages(kvh, page, x16, kv, scales_of):
    """A front tile that holds a few first tokens, a gap, and a window that begins
    inside a tile; and first tokens whose tile the window's begins in."""
    fda = lib()
    for window, sinks, ctx in ((300, 5, [1500, 700, 40]), (100, 3, [230, 250, 900])):
        if page == 128 and window == 100:
            ctx = [400, 250, 900]
        bt = ref.Batch([1, 1, 1], ctx, kvh, 128, kv, page, seed=kvh)
        f = _hidden(bt, scales_of, window, sinks, 3)
        q = _queries(bt, 8 * kvh, x16, 1)
        ws = fda.alloc_workspace(3, 8 * kvh, kvh, 128)
        want, wlse = wref.attention(f, q, 8 * kvh, 128 ** -0.5, window, sinks)
        wref.compare(bt, *_decode(fda, f, q, window, sinks, ws), want, wlse, x16)
        _ok(fda, ws)
        bt = ref.Batch([130, 1, 20], ctx, kvh, 128, kv, page, seed=kvh)
        f = _hidden(bt, scales_of, window, sinks, 3)
        q = _queries(bt, 4 * kvh, x16, 1)
        ws = fda.alloc_prefill_workspace(128)
        want, wlse = wref.attention(f, q, 4 * kvh, 128 ** -0.5, window, sinks)
        wref.compare(bt, *_prefill(fda, f, q, window, sinks, ws), want, wlse, x16)
        _ok(fda, ws)


def test_hidden_scales_cost_nothing():
    """A NaN scale behind the window marks no segment for the repair key by key of
    what is not finite: with it the call took 18 times as long (1880 us, 105)."""
    fda = lib()
    i32 = dict(dtype=torch.int32, device=DEV)
    B, n, T, P, KVH, D, W, S = 4, 512, 8192, 16, 8, 128, 1024, 5
    g = torch.Generator(device=DEV).manual_seed(1)
    pages = B * T // P + 1
    k, v = (torch.randint(-127, 128, (pages, P, KVH, D), generator=g, device=DEV, dtype=torch.int8)
            for _ in range(2))
    scales = torch.rand((pages * P, KVH), generator=g, device=DEV) * 0.01 + 0.005
    bad = scales.clone()
    bad[-P:] = float("nan")
    table = torch.arange(B * T // P, **i32).view(B, -1).clone()
    table[:, 1:(T - n - W) // P] = pages - 1      # given away
    q = torch.randn((B * n, 32, D), generator=g, device=DEV).bfloat16()
    args = (q, k, v, torch.arange(B + 1, **i32) * n, torch.full((B,), T, **i32))
    ws = fda.alloc_prefill_workspace(D)
    outs, best = [], []
    for x in (scales, bad):
        times = []
        for _ in range(10):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            out = fda.prefill_attention(*args, block_table=table, k_scales=x, v_scales=x, window=W,
                                        sinks=S, workspace=ws)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        outs.append(out)
        best.append(min(times))
    _ok(fda, ws)
    assert all(torch.equal(x, y) for x, y in zip(*outs))
    assert best[1] < 3 * best[0], best
