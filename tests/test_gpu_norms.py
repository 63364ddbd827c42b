"""GPU tests of the packed append with norms of query and key heads and rotary
positions on several axes, against a plain statement in fp32 operations (bit for
bit) and the formula in 64 bits."""
import math

import numpy as np
import pytest
import torch

import prompt_ref as ref
import window_ref as wref
from gpu_util import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6


def _ok(fda, ws):
    st, info = fda.fd_check_device_error(ws)
    assert st == fda.FD_OK, (fda.fd_status_string(st), info)


def normed(x, w, eps, dtype=torch.float32):
    """[tokens, heads, d] normed in `dtype` operations: the exact sum of squares
    rounded once, then one rounding per operation."""
    x = x.to(dtype)
    if w is None:
        return x
    mean = x.double().square().sum(-1, keepdim=True).to(dtype) * (1.0 / x.shape[-1])
    one = torch.ones((), dtype=dtype)
    return x * (one / (mean + torch.tensor(eps, dtype=torch.float32).to(dtype)).sqrt()) * w.to(dtype)


def turned(x, tab, pos, rot, interleaved, pair_axes=None):
    """pos: [tokens], or [axes, tokens] with the axis of every pair."""
    if pair_axes is None:
        return ref.rotate(x, tab, pos, rot, interleaved, x.dtype)
    half = rot // 2
    p = pos.long()[torch.tensor(pair_axes)].T          # [tokens, pairs]
    i = torch.arange(half)
    own = torch.cat([tab[p, i], tab[p, i + half]], 1)  # a table of the tokens' own rows
    return ref.rotate(x, own, torch.arange(len(own)), rot, interleaved, x.dtype)


def axes_of(kind, rot):
    n = rot // 2
    if kind == "turns":
        return [i % 3 for i in range(n)]
    if kind == "runs":
        return [0 if i < n // 4 else 1 if i < n // 4 + 3 * n // 8 else 2 for i in range(n)]
    if kind == "four":
        return [(i // 4) % 4 for i in range(n)]
    return [0] * n


CASES = [
    # new, ctx, qh, kvh, d, x16, kv, page, scales, rot, interleaved, norms, f32, axes
    ([1, 1, 1], [0, 5, 99], 8, 2, 128, "f16", "e4m3", 16, "tensor", 128, False, "qk", False, None),
    ([33, 0, 7], [0, 3, 64], 4, 1, 64, "f16", "f16", 0, "tensor", 64, False, "qk", True, None),
    ([129, 1], [1, 300], 6, 2, 128, "bf16", "bf16", 64, "tensor", 64, True, "k", False, None),
    ([20, 13], [17, 0], 8, 8, 128, "bf16", "i8", 8, "token", 128, True, "qk", True, None),
    ([20, 13], [17, 0], 8, 8, 64, "f16", "i8", 1, "head", 16, False, "q", False, "runs"),
    ([700], [3], 32, 8, 128, "f16", "e4m3", 0, "token", 96, False, "qk", True, "turns"),
    ([5, 9], [2, 2], 3, 3, 64, "bf16", "e4m3", 256, "head", 32, True, None, False, "four"),
    ([11, 2], [0, 0], 0, 2, 128, "f16", "e4m3", 16, "tensor", 0, False, "k", False, None),
    ([11, 2], [0, 0], 5, 1, 128, "f16", "i8", 16, "token", 0, False, "qk", False, None),
    ([40, 3], [9, 0], 16, 2, 128, "bf16", "bf16", 16, "tensor", 128, True, "q", True, "turns"),
    ([40, 3], [9, 0], 16, 2, 128, "f16", "f16", 0, "tensor", 128, False, None, False, "runs"),
    ([40, 3], [9, 0], 2, 2, 64, "bf16", "i8", 64, "token", 48, True, "qk", False, "runs"),
    ([900, 1], [0, 0], 64, 8, 128, "bf16", "e4m3", 64, "tensor", 64, False, "qk", False, "one"),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_append(case):
    """Every row, code and scale equals the statement's bit for bit; nothing
    else is written."""
    fda = lib()
    new, ctx, qh, kvh, d, x16, kv, page, scales, rot, inter, norms, f32, axes = CASES[case]
    bt = ref.Batch(new, ctx, kvh, d, kv, page, seed=case, lead=3, tail=5)
    g = torch.Generator().manual_seed(case)
    dt = ref.T16[x16]
    wide = torch.randn((bt.tokens, qh + 2 * kvh, d), generator=g)
    # rows far apart in size, and rows of zeros
    wide *= 10.0 ** torch.randint(-3, 3, (bt.tokens, qh + 2 * kvh, 1), generator=g)
    wide = wide.to(dt)
    wide[int(bt.q_start[0]), qh:] = 0
    gw = wide.to(DEV)
    wt = torch.float32 if f32 else dt
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(wt) if norms and x in norms else None
              for x in "qk")
    kc, vc = (ref.poison(kv, bt.shape()).to(DEV) for _ in range(2))
    scale = 5.0 / ref.QMAX.get(kv, 5.0)
    fine = None
    if scales == "head":
        fine = torch.rand(kvh, generator=g) + 0.5
    elif scales == "token":
        fine = torch.full((bt.rows, kvh), -1.0)
    reach = max(bt.seq)
    ap = pair_axes = None
    if axes:
        pair_axes = axes_of(axes, rot)
        reach = 77
        # a slice of a longer buffer: rows further apart than the tokens
        room = torch.randint(0, reach, (max(pair_axes) + 1, bt.tokens + 9), generator=g,
                             dtype=torch.int32)
        room[:, 0] = -5                      # of nobody
        ap = room.to(DEV)[:, :bt.tokens]
    tab = fda.rotary_table(reach, rot) if rot else None
    q_out = torch.full((bt.tokens, qh, d), 9.0, dtype=dt, device=DEV) if qh else None
    ksc = fine.to(DEV) if fine is not None else None
    vsc = fine.to(DEV).clone() if fine is not None else None
    ws = fda.alloc_prefill_workspace(d)
    res = fda.append_kv(gw[:, qh:qh + kvh], gw[:, qh + kvh:], kc, vc,
                        torch.from_numpy(bt.q_start).to(DEV),
                        torch.tensor(ctx, dtype=torch.int32, device=DEV),
                        q=gw[:, :qh] if qh else None, q_out=q_out, rotary=tab, interleaved=inter,
                        k_scale=scale, v_scale=scale, k_scales=ksc, v_scales=vsc, workspace=ws,
                        q_norm=wq.to(DEV) if wq is not None else None,
                        k_norm=wk.to(DEV) if wk is not None else None, norm_eps=EPS,
                        axis_positions=ap, pair_axes=pair_axes, **bt.index(DEV))
    torch.cuda.synchronize()
    _ok(fda, ws)
    assert res is q_out
    at = torch.cat([torch.arange(n) + int(bt.q_start[b]) for b, n in enumerate(new)])
    where = torch.cat([torch.arange(c, c + n) for n, c in zip(new, ctx)])
    rows = torch.cat([bt.rows_of(b, c, c + n) for b, (n, c) in enumerate(zip(new, ctx))])
    if axes:
        where = ap.cpu()[:, at]
    host = tab.cpu() if rot else None
    v = wide[at][:, qh + kvh:].float()

    def made(x, w, dtype):
        y = normed(x, w, EPS, dtype)
        return turned(y, host, where, rot, inter, pair_axes) if rot else y

    k = made(wide[at][:, qh:qh + kvh], wk, torch.float32)
    for x, cache, fresh in ((k, kc, ksc), (v, vc, vsc)):
        codes, tok = ref.quantise(x, kv, scale, fine, scales)
        want = ref.poison(kv, (bt.rows, kvh, d))
        want[rows] = codes
        assert torch.equal(want.view(torch.uint8),
                           cache.cpu().view(bt.rows, kvh, d).view(torch.uint8))
        if scales == "token":
            full = torch.full((bt.rows, kvh), -1.0)
            full[rows] = tok
            assert torch.equal(full, fresh.cpu())
    if qh:
        want = torch.full((bt.tokens, qh, d), 9.0, dtype=dt)
        want[at] = made(wide[at][:, :qh], wq, torch.float32).to(dt)
        assert torch.equal(want.view(torch.int16), q_out.cpu().view(torch.int16))
        # and the formula in 64 bits: at most ten fp32 roundings (2^-24 each) of
        # values up to the pair's norm, and the rounding to 16 bits; below the
        # type's smallest normal number its step is fixed
        exact = made(wide[at][:, :qh], wq, torch.float64)
        eps, tiny = torch.finfo(dt).eps, torch.finfo(dt).smallest_normal
        mag = exact.abs().amax(-1, keepdim=True)
        tol = eps / 2 * exact.abs() + 20 * 2.0 ** -24 * mag + tiny * eps / 2
        assert torch.all((q_out.double().cpu()[at] - exact).abs() <= tol)


def test_rows_at_the_ends_of_the_range():
    """Zeros stay zeros; the largest and smallest elements, NaN and infinities
    do what the fp32 formula says."""
    fda = lib()
    for dt, top, low in ((torch.float16, 65504.0, 2.0 ** -24), (torch.bfloat16, 1e18, 1e-30),
                         (torch.bfloat16, 3e38, 1e-38)):
        q = torch.zeros((6, 1, 64), dtype=dt)
        q[1] = top
        q[2] = low
        q[3, 0, 5] = float("nan")
        q[4, 0, 6] = float("inf")
        q[5, 0, ::2], q[5, 0, 1::2] = top, -low
        k = torch.zeros((6, 1, 64), dtype=dt)
        kc, vc = (torch.zeros((6, 1, 64), dtype=dt, device=DEV) for _ in range(2))
        i32 = dict(dtype=torch.int32, device=DEV)
        w = torch.ones(64, device=DEV)
        got = fda.append_kv(k.to(DEV), k.to(DEV), kc, vc, torch.tensor([0, 6], **i32),
                            torch.zeros(1, **i32), q=q.to(DEV), q_norm=w, k_norm=w,
                            kv_start_idx=torch.zeros(1, **i32)).cpu()
        want = normed(q.float(), torch.ones(64), EPS)
        if top > 1e30:   # squares past fp32's range: an infinite sum
            for r in (1, 5):
                want[r] = 0
        want = want.to(dt)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        fin = ~torch.isnan(want)
        assert torch.equal(got[fin].abs(), want[fin].abs())
        assert torch.all(kc == 0)


@pytest.mark.parametrize("wt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("at", [1, 2, 3])
def test_weights_inside_a_larger_array(wt, at):
    """Weights that start at any element give what the same ones by themselves do."""
    fda = lib()
    bt = ref.Batch([9, 40], [0, 3], 2, 128, "bf16", 16, seed=5)
    g = torch.Generator().manual_seed(at)
    q, k = (torch.randn((bt.tokens, h, 128), generator=g).to(torch.bfloat16).to(DEV)
            for h in (4, 2))
    room = torch.randn((2, 128 + at), generator=g).to(wt).to(DEV)
    wq, wk = room.reshape(-1)[at:at + 128], room.reshape(-1)[at + 128:at + 256]
    assert wq.data_ptr() % 16 == at * wt.itemsize
    got = []
    for a, b in ((wq, wk), (wq.clone(), wk.clone())):
        kc, vc = (torch.zeros(bt.shape(), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        ws = fda.alloc_prefill_workspace(128)
        out = fda.append_kv(k, k, kc, vc, torch.from_numpy(bt.q_start).to(DEV),
                            torch.tensor([0, 3], dtype=torch.int32, device=DEV), q=q,
                            q_norm=a, k_norm=b, workspace=ws, **bt.index(DEV))
        _ok(fda, ws)
        got.append((out, kc, vc))
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_in_place_queries():
    fda = lib()
    g = torch.Generator().manual_seed(1)
    q = torch.randn((300, 24, 128), generator=g).bfloat16().to(DEV)
    k = torch.randn((300, 4, 128), generator=g).bfloat16().to(DEV)
    kc, vc = (torch.zeros((300, 4, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    i32 = dict(dtype=torch.int32, device=DEV)
    tab = fda.rotary_table(300, 128)
    w = (torch.rand(128, generator=g) + 0.5).to(DEV)
    args = (k, k, kc, vc, torch.tensor([0, 300], **i32), torch.zeros(1, **i32))
    kw = dict(rotary=tab, q_norm=w, k_norm=w, kv_start_idx=torch.zeros(1, **i32))
    want = fda.append_kv(*args, q=q, **kw)
    got = fda.append_kv(*args, q=q, q_out=q, **kw)
    assert got is q and torch.equal(got, want)


def test_positions_outside_the_table():
    """A token with a position outside the table on some axis is left alone and
    recorded; its place in the sequence may lie past the table."""
    fda = lib()
    i32 = dict(dtype=torch.int32, device=DEV)
    ws = fda.alloc_prefill_workspace(64)
    k = torch.ones((4, 1, 64), dtype=torch.float16, device=DEV)
    tab = fda.rotary_table(10, 16)
    for bad, at in ((10, (1, 2)), (-1, (0, 2)), (1 << 30, (2, 2))):
        kc, vc = (torch.zeros((100, 1, 64), dtype=torch.float16, device=DEV) for _ in range(2))
        q_out = torch.zeros((4, 2, 64), dtype=torch.float16, device=DEV)
        ap = torch.full((3, 4), 9, **i32)
        ap[at] = bad
        fda.append_kv(k, k, kc, vc, torch.tensor([0, 4], **i32), torch.tensor([50], **i32),
                      q=torch.ones((4, 2, 64), dtype=torch.float16, device=DEV), q_out=q_out,
                      rotary=tab, axis_positions=ap, pair_axes=[0, 1, 2, 0, 1, 2, 0, 1],
                      kv_start_idx=torch.zeros(1, **i32), workspace=ws)
        torch.cuda.synchronize()
        # (the error word holds value + 1, with 0 for none: -1 reads as 0)
        assert fda.fd_check_device_error(ws) == (fda.FD_ERR_DEVICE_BOUNDS, 0 if bad == -1 else bad)
        assert vc[:, 0, 0].nonzero().flatten().tolist() == [50, 51, 53]
        assert q_out[:, 0, 40].tolist() == [1, 1, 0, 1]


def test_the_prompt_call_norms_and_turns_on_axes():
    """prefill_attention with new keys, norms, axes and a window: the caches and
    outputs of the separate calls; queries without a table are normed too."""
    fda = lib()
    bt = ref.Batch([40, 1, 9], [3, 90, 0], 2, 64, "e4m3", 16, seed=5)
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn((bt.tokens, h, 64), generator=g).half().to(DEV) for h in (8, 2, 2))
    w = [(torch.rand(64, generator=g) + 0.5).half().to(DEV) for _ in range(2)]
    i32 = dict(dtype=torch.int32, device=DEV)
    qs, seq = torch.from_numpy(bt.q_start).to(DEV), torch.tensor(bt.seq, **i32)
    pos = torch.tensor(bt.ctx, **i32)
    ap = torch.randint(0, 30, (3, bt.tokens), generator=g, dtype=torch.int32).to(DEV)
    at = dict(k_scale=0.03, v_scale=0.03, **bt.index(DEV))
    for rotary, axes in ((fda.rotary_table(30, 64), dict(axis_positions=ap, pair_axes=axes_of("runs", 64))),
                         (fda.rotary_table(100, 64), {}), (None, {})):
        caches = [torch.full(bt.shape(), 0x38, dtype=torch.uint8, device=DEV) for _ in range(4)]
        norm = dict(rotary=rotary, q_norm=w[0], k_norm=w[1], norm_eps=1e-5, **axes)
        one = fda.prefill_attention(q, caches[0], caches[1], qs, seq, k_new=k, v_new=v,
                                    positions=pos, window=20, sinks=2, **norm, **at)
        q2 = fda.append_kv(k, v, caches[2], caches[3], qs, pos, q=q, **norm, **at)
        two = fda.prefill_attention(q2, caches[2], caches[3], qs, seq, window=20, sinks=2, **at)
        torch.cuda.synchronize()
        assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
        assert not torch.equal(q2, q)


def test_a_step_without_tokens():
    """Norms, axes and a window with nothing to do: empty results, caches as they were."""
    fda = lib()
    kc, vc = (torch.full((16, 2, 64), 3.0, dtype=torch.float16, device=DEV) for _ in range(2))
    q, k = (torch.zeros((0, h, 64), dtype=torch.float16, device=DEV) for h in (4, 2))
    w, tab = torch.ones(64, dtype=torch.float16, device=DEV), fda.rotary_table(16, 32)
    i32 = dict(dtype=torch.int32, device=DEV)
    starts, zeros = torch.zeros(3, **i32), torch.zeros(2, **i32)
    kw = dict(q_norm=w, k_norm=w, rotary=tab, axis_positions=torch.zeros((2, 0), **i32),
              pair_axes=[0, 1] * 8, kv_start_idx=torch.tensor([0, 8], **i32))
    assert fda.append_kv(k, k, kc, vc, starts, zeros, q=q, **kw).shape == (0, 4, 64)
    for window in (None, 5):
        out, lse = fda.prefill_attention(q, kc, vc, starts, zeros, k_new=k, v_new=k,
                                         positions=zeros, window=window, **kw)
        assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    assert torch.all(kc == 3) and torch.all(vc == 3)


def test_append_in_a_graph_and_on_another_stream():
    fda = lib()
    n, i32 = 50, dict(dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(2)
    q, k = torch.zeros((n, 8, 128), device=DEV).half(), torch.zeros((n, 2, 128), device=DEV).half()
    kc, vc = (torch.zeros((n, 2, 128), dtype=torch.int8, device=DEV) for _ in range(2))
    ap = torch.zeros((2, n), **i32)
    w = (torch.rand(128, generator=g) + 0.5).to(DEV)
    tab = fda.rotary_table(64, 128)
    axes = [i % 2 for i in range(64)]
    start, zero = torch.tensor([0, n], **i32), torch.zeros(1, **i32)
    ws = fda.alloc_prefill_workspace(128)
    out = torch.zeros_like(q)

    def call(**kw):
        fda.append_kv(k, k, kc, vc, start, zero, q=q, q_out=out, rotary=tab, q_norm=w, k_norm=w,
                      axis_positions=ap, pair_axes=axes, kv_start_idx=zero, k_scale=0.03,
                      v_scale=0.03, workspace=ws, **kw)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in range(2):
        g.manual_seed(10 + seed)
        hq, hk = torch.randn(q.shape, generator=g).half(), torch.randn(k.shape, generator=g).half()
        hp = torch.randint(0, 64, ap.shape, generator=g, dtype=torch.int32)
        q.copy_(hq)
        k.copy_(hk)
        ap.copy_(hp)
        graph.replay()
        torch.cuda.synchronize()
        host = tab.cpu()
        want = turned(normed(hq, w.cpu(), EPS), host, hp, 128, False, axes).half()
        assert torch.equal(out.cpu(), want)
        kk = turned(normed(hk, w.cpu(), EPS), host, hp, 128, False, axes)
        codes, _ = ref.quantise(kk, "i8", 0.03, None, "tensor")
        assert torch.equal(kc.cpu(), codes)
