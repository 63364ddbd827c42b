"""GPU tests of the prompt path (rotary table, packed append, read-back,
attention of packed new tokens) against plain 64-bit statements."""
import math

import numpy as np
import pytest
import torch

import prompt_ref as ref
from gpu_util import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _ok(fda, ws):
    st, info = fda.fd_check_device_error(ws)
    assert st == fda.FD_OK, (fda.fd_status_string(st), info)


# ---------------------------------------------------------------------------
# rotary table
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("positions,rot,theta,scaling,factor,amplitude", [
    (1, 16, 10000.0, "none", 1.0, 1.0),
    (7, 128, 10000.0, "none", 1.0, 1.0),
    (4097, 64, 10000.0, "linear", 4.0, 1.0),
    (1001, 48, 500000.0, "by_parts", 8.0, 1.25),
    (131072, 128, 1000000.0, "none", 1.0, 1.0),
])
def test_rotary_table(positions, rot, theta, scaling, factor, amplitude):
    fda = lib()
    got = fda.rotary_table(positions, rot, theta=theta, scaling=scaling, factor=factor,
                           original_positions=8192.0, low_turns=1.0, high_turns=32.0,
                           amplitude=amplitude).double().cpu().numpy()
    want = ref.table(positions, rot, theta, scaling, factor, 8192.0, 1.0, 32.0, amplitude)
    # fp32: the reduced angle carries two roundings (conversion, times 2 pi),
    # |y| <= pi/4, so at most pi/2 * 2^-24 into cos or sin; the last sum and
    # the amplitude round once each (2^-24 each), the earlier terms of the
    # sums less than another 2^-24 together.  The reference's own angle
    # p * f is good to p * 2^-52.
    tol = amplitude * (math.pi / 2 + 3) * 2.0 ** -24 + positions * 2.0 ** -52
    assert np.abs(got - want).max() <= tol
    # row 0: no rotation, exactly
    assert np.all(got[0, :rot // 2] == np.float32(amplitude)) and np.all(got[0, rot // 2:] == 0)


def test_rotary_table_keeps_small_angles_and_a_given_buffer():
    fda = lib()
    buf = torch.full((3, 128), 7.0, device=DEV)
    out = fda.rotary_table(3, 128, theta=1e8, out=buf)
    assert out is buf
    want = ref.table(3, 128, 1e8)
    got = buf.double().cpu().numpy()
    # sines of angles below 1e-7 keep their relative accuracy
    rel = np.abs(got[1:, 64:] - want[1:, 64:]) / np.abs(want[1:, 64:])
    assert rel.max() <= 4 * 2.0 ** -24


# ---------------------------------------------------------------------------
# packed append
# ---------------------------------------------------------------------------

APPEND = [
    # new, ctx, qh, kvh, d, x16, kv, page, scales, rot, interleaved
    ([1, 1, 1], [0, 5, 99], 8, 2, 128, "f16", "e4m3", 16, "tensor", 128, False),
    ([33, 0, 7], [0, 3, 64], 4, 1, 64, "f16", "f16", 0, "tensor", 64, False),
    ([129, 1], [1, 300], 6, 2, 128, "bf16", "bf16", 64, "tensor", 64, True),
    ([20, 13], [17, 0], 8, 8, 128, "bf16", "i8", 8, "token", 128, True),
    ([20, 13], [17, 0], 8, 8, 64, "f16", "i8", 1, "head", 16, False),
    ([700], [3], 32, 8, 128, "f16", "e4m3", 0, "token", 96, False),
    ([5, 9], [2, 2], 3, 3, 64, "bf16", "e4m3", 256, "head", 32, True),
    ([11, 2], [0, 0], 0, 2, 128, "f16", "e4m3", 16, "tensor", 0, False),
]


@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_packed(case):
    """Every row, code and scale equals the statement's bit for bit; nothing
    else is written, in the caches or in the packed arrays."""
    fda = lib()
    new, ctx, qh, kvh, d, x16, kv, page, scales, rot, inter = APPEND[case]
    bt = ref.Batch(new, ctx, kvh, d, kv, page, seed=case, lead=3, tail=5)
    g = torch.Generator().manual_seed(case)
    dt = ref.T16[x16]
    # one projection's output: q, k and v side by side in a token's row
    wide = torch.randn((bt.tokens, qh + 2 * kvh, d), generator=g).to(dt)
    wide[int(bt.q_start[0]), qh:] = 0                  # a row of zeros: scale 1
    gw = wide.to(DEV)
    kc, vc = (ref.poison(kv, bt.shape()).to(DEV) for _ in range(2))
    scale = 5.0 / ref.QMAX.get(kv, 5.0)
    fine = None
    if scales == "head":
        fine = torch.rand(kvh, generator=g) + 0.5
    elif scales == "token":
        fine = torch.full((bt.rows, kvh), -1.0)
    tab = fda.rotary_table(400 if rot else 1, rot or 16)[:max(bt.seq)] if rot else None
    if rot and tab.shape[0] < max(bt.seq):
        tab = fda.rotary_table(max(bt.seq), rot)
    q_out = torch.full((bt.tokens, qh, d), 9.0, dtype=dt, device=DEV) if qh else None
    ksc = fine.to(DEV) if fine is not None else None
    vsc = fine.to(DEV).clone() if fine is not None else None
    ws = fda.alloc_prefill_workspace(d)
    pos = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    res = fda.append_kv(gw[:, qh:qh + kvh], gw[:, qh + kvh:], kc, vc,
                        torch.from_numpy(bt.q_start).to(DEV), pos, q=gw[:, :qh] if qh else None,
                        q_out=q_out, rotary=tab, interleaved=inter, k_scale=scale, v_scale=scale,
                        k_scales=ksc, v_scales=vsc, workspace=ws, **bt.index(DEV))
    torch.cuda.synchronize()
    _ok(fda, ws)
    assert res is q_out
    # the statement, in fp32 operations
    at = torch.cat([torch.arange(n) + int(bt.q_start[b]) for b, n in enumerate(new)])
    where = torch.cat([torch.arange(c, c + n) for n, c in zip(new, ctx)])
    rows = torch.cat([bt.rows_of(b, c, c + n) for b, (n, c) in enumerate(zip(new, ctx))])
    q, k, v = wide[at][:, :qh], wide[at][:, qh:qh + kvh].float(), wide[at][:, qh + kvh:].float()
    if rot:
        host = tab.cpu()
        q = ref.rotate(q, host, where, rot, inter, torch.float32).to(dt)
        k = ref.rotate(k, host, where, rot, inter, torch.float32)
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
        want[at] = q
        assert torch.equal(want.view(torch.int16), q_out.cpu().view(torch.int16))


def test_append_agrees_with_the_decode_append():
    """A step of one token per sequence, without a table, leaves the caches
    that fd_append_kv leaves."""
    fda = lib()
    bt = ref.Batch([1] * 5, [0, 1, 17, 40, 3], 2, 128, "i8", 16, seed=4)
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn((5, 2, 128), generator=g).half().to(DEV) for _ in range(2))
    pos = torch.tensor(bt.ctx, dtype=torch.int32, device=DEV)
    got = []
    for packed in (False, True):
        kc, vc = (torch.zeros(bt.shape(), dtype=torch.int8, device=DEV) for _ in range(2))
        ks, vs = (torch.zeros((bt.rows, 2), device=DEV) for _ in range(2))
        ix = bt.index(DEV)
        if packed:
            fda.append_kv(k, v, kc, vc, torch.arange(6, dtype=torch.int32, device=DEV), pos,
                          k_scale=0.5, v_scale=2.0, k_scales=ks, v_scales=vs, **ix)
        else:
            fda.fd_append_kv(k, v, kc, vc, None, ix["block_table"], pos, bt.rows, 2, 128, 16, 0.5,
                             2.0, fda.FD_SCALE_TOKEN, ks, vs, fda.alloc_workspace(5, 2, 2, 128))
        got.append([x.cpu() for x in (kc, vc, ks, vs)])
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_append_leaves_and_records():
    """A negative position leaves a sequence alone; tokens past the table, the
    block table's row or the cache are skipped and recorded."""
    fda = lib()
    d, kvh = 64, 1
    ws = fda.alloc_prefill_workspace(d)
    k = torch.ones((6, kvh, d), dtype=torch.float16, device=DEV)
    qs = torch.tensor([0, 3, 6], dtype=torch.int32, device=DEV)

    def call(pos, rotary=None, bt=((0, 1), (2, 3))):
        kc, vc = (torch.zeros((4, 2, kvh, d), dtype=torch.float16, device=DEV) for _ in range(2))
        q_out = torch.zeros((6, 2, d), dtype=torch.float16, device=DEV)
        fda.append_kv(k, k, kc, vc, qs, torch.tensor(pos, dtype=torch.int32, device=DEV),
                      q=torch.ones((6, 2, d), dtype=torch.float16, device=DEV), q_out=q_out,
                      rotary=rotary, block_table=torch.tensor(bt, dtype=torch.int32, device=DEV),
                      workspace=ws)
        torch.cuda.synchronize()
        st, info = fda.fd_check_device_error(ws)
        return (kc.view(8, d)[:, 0].cpu().tolist(), q_out[:, 0, 0].cpu().tolist(), st, info)

    assert call([-1, 0]) == ([0, 0, 0, 0, 1, 1, 1, 0], [0, 0, 0, 1, 1, 1], fda.FD_OK, 0)
    rows, q, st, info = call([2, 0])            # tokens 2..4 of four: one past the row
    assert rows == [0, 0, 1, 1, 1, 1, 1, 0] and q[2] == 0 and (st, info) == (5, 4)
    rows, q, st, info = call([0, 0], bt=((0, 9), (-3, 3)))
    assert rows == [1, 1, 0, 0, 0, 0, 1, 0] and st == 5 and info in (9, -3)
    tab = fda.rotary_table(2, 16)
    rows, q, st, info = call([0, 1], rotary=tab)
    assert rows[:4] == [1, rows[1], 0, 0] and q[2] == 0 and st == 5 and info in (2, 3)


# ---------------------------------------------------------------------------
# read-back
# ---------------------------------------------------------------------------

READ = [
    ([5, 0, 130], [0, 3, 17], 2, 128, "e4m3", 16, "tensor", "f16"),
    ([1], [0], 1, 64, "i8", 0, "token", "bf16"),
    ([77, 3], [0, 500], 8, 128, "i8", 64, "token", "f16"),
    ([40, 41, 1], [1, 0, 9], 3, 64, "e4m3", 1, "head", "bf16"),
    ([9, 200], [2, 2], 5, 128, "bf16", 8, "tensor", "bf16"),
    ([64, 65], [0, 0], 1, 64, "f16", 0, "tensor", "f16"),
]


@pytest.mark.parametrize("case", range(len(READ)))
def test_read_back(case):
    fda = lib()
    new, ctx, kvh, d, kv, page, scales, x16 = READ[case]
    bt = ref.Batch(new, ctx, kvh, d, kv, page, seed=case, lead=2, tail=3)
    f = ref.Filled(bt, scales, seed=case)
    ws = fda.alloc_prefill_workspace(d)
    kw = f.device(DEV)
    ko, vo = (torch.full((bt.tokens, kvh, d), 9.0, dtype=ref.T16[x16], device=DEV)
              for _ in range(2))
    start = torch.from_numpy(bt.q_start).to(DEV)
    first = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    got = fda.read_kv(kw.pop("k_cache"), kw.pop("v_cache"), start, bt.tokens, first=first,
                      k_out=ko, v_out=vo, workspace=ws, **kw, **bt.index(DEV))
    torch.cuda.synchronize()
    _ok(fda, ws)
    assert got[0] is ko and got[1] is vo
    eps = torch.finfo(ref.T16[x16]).eps
    for w, t in zip("kv", got):
        t = t.double().cpu()
        mine = torch.zeros(bt.tokens, dtype=torch.bool)
        for b, n in enumerate(new):
            i = int(bt.q_start[b])
            mine[i:i + n] = True
            want = f.val[w][bt.rows_of(b, ctx[b], ctx[b] + n)]
            # two fp32 products (2^-24 each) and the rounding to 16 bits: half
            # a step of the value, or below the smallest normal number half of
            # the fixed step there (the smallest e4m3 code times the scale,
            # 2^-9 * 5 / 448 = 2.2e-5, is a subnormal f16: step 2^-24)
            tiny = torch.finfo(ref.T16[x16]).smallest_normal * eps / 2
            tol = want.abs() * (eps / 2 + 2.0 ** -22) + tiny
            assert torch.all((t[i:i + n] - want).abs() <= tol)
        assert torch.all(t[~mine] == 9.0)


def test_read_back_of_what_is_not_there():
    """Rows of tokens outside the cache come back as zeros and are recorded;
    without `first` a sequence is read from its start."""
    fda = lib()
    ws = fda.alloc_prefill_workspace(64)
    k = torch.arange(1, 9, device=DEV, dtype=torch.float16).view(4, 2, 1, 1).expand(4, 2, 1, 64)
    k = k.contiguous()
    bt = torch.tensor([[1, 77], [2, 0]], dtype=torch.int32, device=DEV)
    start = torch.tensor([0, 3, 6], dtype=torch.int32, device=DEV)
    ko, vo = fda.read_kv(k, k, start, 6, block_table=bt, workspace=ws)
    torch.cuda.synchronize()
    assert ko[:, 0, 5].cpu().tolist() == [3, 4, 0, 5, 6, 1]
    assert torch.equal(ko, vo)
    assert fda.fd_check_device_error(ws) == (fda.FD_ERR_DEVICE_BOUNDS, 77)


# ---------------------------------------------------------------------------
# attention of packed new tokens
# ---------------------------------------------------------------------------

ATTN = [
    # new, ctx, qh, kvh, d, x16, kv, page, scales
    ([7, 33], [0, 0], 4, 1, 64, "f16", "f16", 0, "tensor"),
    ([1, 1, 1], [0, 127, 128], 8, 2, 128, "bf16", "bf16", 16, "tensor"),
    ([1], [1], 1, 1, 64, "f16", "f16", 0, "tensor"),
    ([130, 0, 5], [0, 9, 700], 8, 2, 128, "f16", "f16", 64, "tensor"),
    ([300], [0], 2, 2, 128, "bf16", "bf16", 0, "tensor"),
    ([257, 64], [100, 1000], 6, 2, 64, "bf16", "bf16", 8, "tensor"),
    ([40, 3], [333, 0], 10, 2, 128, "f16", "f16", 1, "tensor"),
    ([9, 128], [4, 260], 5, 1, 64, "f16", "f16", 4, "tensor"),
    ([128, 129], [0, 383], 16, 2, 128, "f16", "e4m3", 64, "tensor"),
    ([61, 2], [1000, 255], 8, 8, 128, "bf16", "e4m3", 0, "head"),
    ([100, 1], [29, 2000], 4, 1, 64, "f16", "e4m3", 16, "token"),
    ([77, 1], [0, 515], 8, 1, 128, "f16", "i8", 16, "tensor"),
    ([50, 50], [7, 250], 32, 8, 128, "bf16", "i8", 256, "token"),
    ([19, 200], [0, 5], 12, 12, 64, "bf16", "i8", 2, "head"),
    ([4, 1], [3000, 5000], 128, 1, 128, "f16", "e4m3", 64, "tensor"),
    ([3], [10], 127, 1, 64, "bf16", "bf16", 0, "tensor"),
    ([6, 1], [700, 20], 65, 1, 128, "f16", "i8", 8, "token"),
]


def _attend(fda, f, q, qh, ws, scale=None, **more):
    bt = f.batch
    kw = f.device(DEV)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    fda.prefill_attention(q.to(DEV), kw.pop("k_cache"), kw.pop("v_cache"),
                          torch.from_numpy(bt.q_start).to(DEV),
                          torch.tensor(bt.seq, dtype=torch.int32, device=DEV), out=out, lse=lse,
                          workspace=ws, softmax_scale=scale, **kw, **bt.index(DEV), **more)
    torch.cuda.synchronize()
    return out.double().cpu(), lse.double().cpu()


def _compare(f, out, lse, want, wlse, x16, label=""):
    bt = f.batch
    mine = torch.zeros(out.shape[0], dtype=torch.bool)
    for b, n in enumerate(bt.new):
        mine[int(bt.q_start[b]):int(bt.q_start[b]) + n] = True
    assert torch.all(out[~mine] == 7.0) and torch.all(lse[~mine] == 7.0)
    out, lse, want, wlse = out[mine], lse[mine], want[mine], wlse[mine]
    empty = wlse == -math.inf
    assert torch.equal(lse == -math.inf, empty) and torch.all(out[empty] == 0)
    out, lse, want, wlse = out[~empty], lse[~empty], want[~empty], wlse[~empty]
    if not len(out):
        return
    # A probability and the output are each rounded once to 16 bits (half a
    # step, eps / 2, of the value).  The probabilities' errors reach the
    # output weighted by v: at most eps / 2 * max |v|, with N(0, 1) draws of
    # these sizes below 5.5; the output's own eps / 2 * |out|.  fp32 products,
    # sums and ex2 add a few 2^-22 of the same magnitudes.
    eps = torch.finfo(ref.T16[x16]).eps
    tol = (eps / 2 + 2.0 ** -18) * 5.5 + (eps / 2) * want.abs()
    assert torch.all((out - want).abs() <= tol), (label, float(((out - want).abs() - tol).max()))
    # scores up to about 40 in fp32 (128 products), and ex2 / lg2
    assert float((lse - wlse).abs().max()) <= 1e-4 * max(1.0, float(wlse.abs().max())), label
    rel = float(torch.linalg.norm(out - want) / torch.linalg.norm(want))
    assert rel <= eps, (label, rel)     # two independent roundings: sqrt(2) eps / sqrt(12) rms


@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention(case):
    fda = lib()
    new, ctx, qh, kvh, d, x16, kv, page, scales = ATTN[case]
    bt = ref.Batch(new, ctx, kvh, d, kv, page, seed=case, lead=2, tail=3)
    f = ref.Filled(bt, scales, seed=case)
    q = torch.randn((bt.tokens, qh, d), generator=torch.Generator().manual_seed(case))
    q = q.to(ref.T16[x16])
    ws = fda.alloc_prefill_workspace(d)
    out, lse = _attend(fda, f, q, qh, ws)
    _ok(fda, ws)
    want, wlse = ref.attention(f, q, qh, d ** -0.5)
    _compare(f, out, lse, want, wlse, x16, str(ATTN[case]))


def test_attention_rows_without_keys():
    """Sequences shorter than their packed tokens: the first tokens have no
    key; an empty sequence has none at all."""
    fda = lib()
    bt = ref.Batch([200, 3, 5, 40], [-190, -3, -2, 10], 2, 64, "bf16", 16, seed=3)
    f = ref.Filled(bt, seed=3)
    q = torch.randn((bt.tokens, 4, 64), generator=torch.Generator().manual_seed(3)).bfloat16()
    ws = fda.alloc_prefill_workspace(64)
    out, lse = _attend(fda, f, q, 4, ws)
    _ok(fda, ws)
    want, wlse = ref.attention(f, q, 4, 64 ** -0.5)
    assert int((wlse == -math.inf).sum()) == 4 * (190 + 3 + 2)
    _compare(f, out, lse, want, wlse, "bf16")
