"""GPU tests of the prompt path (rotary table, packed append, read-back,
attention of packed new tokens) against plain 64-bit statements."""
import math
import threading

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


@pytest.mark.parametrize("positions,rot", [(2432, 128), (2433, 128), (38913, 128), (320007, 128),
                                           (155649, 16), (25537, 96)])
def test_rotary_table_in_many_steps(positions, rot):
    """Tables of one step, of several and of more blocks than fit at once, with
    ends inside a step; every 61st row and the last ones."""
    fda = lib()
    got = fda.rotary_table(positions, rot, theta=1e6)
    at = torch.cat([torch.arange(0, positions, 61), torch.arange(positions - 40, positions)])
    f = 1e6 ** (-2 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    x = at.double()[:, None] * f
    want = torch.cat([x.cos(), x.sin()], dim=1)
    # as above (its bound covers the two levels of sums too: 4.43 * 2^-24); the
    # angles of this statement are good to p * 2^-52 (f) and p * 2^-53 (product)
    tol = (math.pi / 2 + 3) * 2.0 ** -24 + positions * 2.0 ** -51
    assert (got[at.to(DEV)].double().cpu() - want).abs().max().item() <= tol


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


def _queries(bt, qh, x16, seed, scale=1.0):
    q = torch.randn((bt.tokens, qh, bt.d), generator=torch.Generator().manual_seed(seed)) * scale
    return q.to(ref.T16[x16])


@pytest.mark.parametrize("seed", range(24))
def test_attention_many_streams(seed):
    """Random batches of many sequences, so that a CTA passes several streams
    (with rows in one or both of its query tiles, whole and cut) one after the
    other: every format, layout, scale kind and head grouping."""
    fda = lib()
    rng = np.random.default_rng(1000 + seed)
    kvh, group = [(8, 1), (2, 8), (1, 16), (4, 3), (8, 4), (3, 5)][seed % 6]
    d = 64 if seed % 4 else 128
    x16 = ["f16", "bf16"][seed % 2]
    kv = [x16, "e4m3", "i8"][(seed // 2) % 3]
    scales = ["tensor", "head", "token"][(seed // 6) % 3] if kv in ref.QMAX else "tensor"
    page = [0, 16, 64, 4, 256, 8][(seed // 3) % 6]
    B = int(rng.integers(30, 90))
    new = [int(x) for x in rng.choice([0, 1, 1, 2, 17, 40, 90], B)]
    ctx = [int(x) for x in rng.choice([0, 0, 1, 100, 127, 128, 300, -1], B)]
    new[0], ctx[0] = 200, 40
    ctx = [max(c, -n) for n, c in zip(new, ctx)]
    bt = ref.Batch(new, ctx, kvh, d, kv, page, seed=seed, lead=1, tail=2)
    f = ref.Filled(bt, scales, seed=seed)
    q = _queries(bt, kvh * group, x16, seed)
    ws = fda.alloc_prefill_workspace(d)
    out, lse = _attend(fda, f, q, kvh * group, ws)
    _ok(fda, ws)
    want, wlse = ref.attention_blocks(f, q, kvh * group, d ** -0.5)
    _compare(f, out, lse, want, wlse, x16, f"{kvh}x{group} d{d} {x16}/{kv} {scales} page {page}")
    # the same bits again: nothing depends on the order CTAs run in
    again, lagain = _attend(fda, f, q, kvh * group, ws)
    assert torch.equal(out, again) and torch.equal(lse, lagain)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 2.0])
@pytest.mark.parametrize("kv,scales", [("f16", "tensor"), ("e4m3", "token"), ("i8", "head")])
def test_attention_score_scales(scale, kv, scales):
    """Negative, zero and large softmax scales (the running maximum moves and
    the accumulator is rescaled)."""
    fda = lib()
    bt = ref.Batch([70, 300, 1], [0, 500, 900], 2, 128, kv, 16, seed=5)
    f = ref.Filled(bt, scales, seed=5)
    q = _queries(bt, 8, "f16", 5)
    ws = fda.alloc_prefill_workspace(128)
    out, lse = _attend(fda, f, q, 8, ws, scale=scale)
    _ok(fda, ws)
    want, wlse = ref.attention_blocks(f, q, 8, scale)
    _compare(f, out, lse, want, wlse, "f16")


def test_attention_value_scales_over_a_wide_range():
    """Per-token V scales from 1e-7 to 1e5 with f16 queries: their exponents
    are carried beside P."""
    fda = lib()
    bt = ref.Batch([40, 3], [500, 900], 2, 64, "i8", 16, seed=6)
    f = ref.Filled(bt, "token", seed=6)
    owned = ~torch.isnan(f.kw["v_scales"])
    g = torch.Generator().manual_seed(9)
    mag = 10.0 ** (torch.rand(f.kw["v_scales"].shape, generator=g) * 12 - 7)
    old = f.kw["v_scales"].clone()
    f.kw["v_scales"][owned] = mag[owned]
    f.val["v"] = f.val["v"] * (f.kw["v_scales"].double() / old.double())[:, :, None]
    q = _queries(bt, 4, "f16", 6)
    # outputs far beyond f16: the caller's v_scale brings them back
    f.kw["v_scale"] = f.kw["v_scale"] * 1e-3
    f.val["v"] = f.val["v"] * 1e-3
    ws = fda.alloc_prefill_workspace(64)
    out, lse = _attend(fda, f, q, 4, ws)
    _ok(fda, ws)
    want, wlse = ref.attention_blocks(f, q, 4, 64 ** -0.5)
    # P is rounded to f16 (half a step: 2^-11 of itself) against the largest
    # value seen, and the output once more
    top = float(f.val["v"].abs().nan_to_num().max())
    mine = ~torch.isnan(wlse)
    assert torch.all((out - want)[mine].abs() <= 2.0 ** -11 * (top + want[mine].abs()))
    assert float((lse - wlse)[mine].abs().max()) <= 1e-4


@pytest.mark.parametrize("kv,page", [("bf16", 0), ("f16", 16), ("bf16", 4), ("e4m3", 16),
                                     ("e4m3", 0), ("e4m3", 2)])
def test_attention_nonfinite_values_stay_with_their_readers(kv, page):
    """NaN and infinite V elements of new tokens reach the tokens that see
    them, and no other; unseen K rows may hold anything."""
    fda = lib()
    x16 = kv if kv in ref.T16 else "f16"
    bt = ref.Batch([90, 300, 30], [20, 0, 400], 2, 64, kv, page, seed=7)
    f = ref.Filled(bt, seed=7)
    q = _queries(bt, 4, x16, 7)
    marks = [(0, 60, 0, 5, float("nan")), (1, 100, 1, 9, float("inf")), (1, 200, 1, 9, -math.inf),
             (1, 130, 0, 63, float("inf")), (2, 415, 1, 0, float("nan"))]
    for b, t, h, dim, x in marks:
        row = bt.row(b, t)
        if kv == "e4m3":
            x = float("nan")
            f.kw["v_cache"].view(bt.rows, 2, 64)[row, h, dim] = 0x7F
        else:
            f.kw["v_cache"].view(bt.rows, 2, 64)[row, h, dim] = x
        f.val["v"][row, h, dim] = x
    # the last token of each sequence has NaN keys: nobody before it sees them
    for b, T in enumerate(bt.seq):
        row = bt.row(b, T - 1)
        f.kw["k_cache"].view(bt.rows, 2, 64)[row] = 0x7F if kv == "e4m3" else float("nan")
    ws = fda.alloc_prefill_workspace(64)
    out, lse = _attend(fda, f, q, 4, ws)
    _ok(fda, ws)
    want, wlse = ref.attention(f, q, 4, 64 ** -0.5)
    for b, T in enumerate(bt.seq):
        i, n = int(bt.q_start[b]), bt.new[b]
        assert torch.isnan(out[i + n - 1]).all() and torch.isnan(lse[i + n - 1]).all()
        o, w = out[i:i + n - 1], want[i:i + n - 1]
        assert torch.equal(torch.isnan(o), torch.isnan(w)), b
        assert torch.equal(torch.isinf(o), torch.isinf(w)) and torch.equal(o[torch.isinf(o)],
                                                                           w[torch.isinf(w)])
        fin = torch.isfinite(w)
        eps = torch.finfo(ref.T16[x16]).eps
        assert torch.all((o - w)[fin].abs() <= (eps / 2 + 2.0 ** -18) * 5.5 + eps / 2 * w[fin].abs())


def test_attention_nan_scales_of_unseen_keys():
    """A later token's per-token scales may be NaN."""
    fda = lib()
    for x16 in ("f16", "bf16"):
        bt = ref.Batch([150, 3], [10, 200], 1, 64, "i8", 16, seed=8)
        f = ref.Filled(bt, "token", seed=8)
        for b, T in enumerate(bt.seq):
            f.kw["k_scales"][bt.row(b, T - 1)] = float("nan")
            f.kw["v_scales"][bt.row(b, T - 1)] = float("nan")
        q = _queries(bt, 4, x16, 8)
        ws = fda.alloc_prefill_workspace(64)
        out, lse = _attend(fda, f, q, 4, ws)
        want, wlse = ref.attention_blocks(f, q, 4, 64 ** -0.5)
        eps = torch.finfo(ref.T16[x16]).eps
        for b in range(2):
            i, n = int(bt.q_start[b]), bt.new[b]
            o, w = out[i:i + n - 1], want[i:i + n - 1]
            assert torch.all((o - w).abs() <= (eps / 2 + 2.0 ** -18) * 5.5 + eps / 2 * w.abs())
            assert torch.isnan(out[i + n - 1]).all()


def test_attention_strided_queries_and_no_lse():
    fda = lib()
    bt = ref.Batch([33, 7], [0, 50], 2, 128, "bf16", 0, seed=9)
    f = ref.Filled(bt, seed=9)
    wide = torch.randn((40, 12, 128), generator=torch.Generator().manual_seed(9)).bfloat16().to(DEV)
    q = wide[:, 2:10]
    ws = fda.alloc_prefill_workspace(128)
    kw, ix = f.device(DEV), bt.index(DEV)
    qs = torch.from_numpy(bt.q_start).to(DEV)
    sl = torch.tensor(bt.seq, dtype=torch.int32, device=DEV)
    out, lse = fda.prefill_attention(q, kw["k_cache"], kw["v_cache"], qs, sl, workspace=ws, **ix)
    out2, _ = fda.prefill_attention(q.contiguous(), kw["k_cache"], kw["v_cache"], qs, sl,
                                    workspace=ws, **ix)
    assert torch.equal(out, out2)
    out3 = torch.empty_like(out2)
    fda.fd_prefill_attention(q, 12 * 128, kw["k_cache"], kw["v_cache"], ix["kv_start_idx"], None,
                             qs, sl, 40, bt.rows, 8, 2, 128, 0, 128 ** -0.5, 1.0, 1.0, 0, None, None,
                             out3, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, out3)


def test_attention_what_lies_outside():
    """A page outside the cache makes its 128-key tile absent and is recorded;
    a sequence whose start entries are wrong is skipped and recorded; the
    other sequences are served."""
    fda = lib()
    bt = ref.Batch([20, 30], [300, 40], 1, 64, "f16", 16, seed=10)
    f = ref.Filled(bt, seed=10)
    q = _queries(bt, 2, "f16", 10)
    ws = fda.alloc_prefill_workspace(64)
    want, wlse = ref.attention_blocks(f, q, 2, 0.125)
    good = bt.block_table.copy()
    for col, bad in ((3, -7), (9, 10 ** 6)):       # keys 48.., 144..
        bt.block_table = good.copy()
        bt.block_table[0, col] = bad
        out, lse = _attend(fda, f, q, 2, ws)
        assert fda.fd_check_device_error(ws) == (fda.FD_ERR_DEVICE_BOUNDS, bad)
        assert torch.allclose(out[20:], want[20:], atol=3e-3)
        # the tile's keys are left out of the others' softmax
        bt.block_table = good
        tile = col * 16 // 128
        keys = [t for t in range(320) if t // 128 != tile]
        rows = torch.tensor([bt.row(0, t) for t in keys])
        for j in (0, 19):
            seen = [i for i, t in enumerate(keys) if t <= 300 + j]
            s = q[j].double() @ f.val["k"][rows[seen], 0].T * 0.125
            w = torch.softmax(s, -1) @ f.val["v"][rows[seen], 0]
            assert torch.allclose(out[j], w, atol=3e-3)
    for starts in ([0, -5, 50], [0, 60, 50], [30, 20, 50]):
        bt.q_start = np.array(starts, np.int32)
        out, lse = _attend(fda, f, q, 2, ws)
        st, info = fda.fd_check_device_error(ws)
        assert st == fda.FD_ERR_DEVICE_BOUNDS and info in starts


def test_attention_timeout_is_reported():
    """A producer that issues nothing: every wait gives up, the timeout is
    recorded, and the next call is right."""
    fda = lib()
    bt = ref.Batch([200, 1], [10, 700], 2, 128, "e4m3", 16, seed=11)
    f = ref.Filled(bt, seed=11)
    q = _queries(bt, 8, "f16", 11)
    ws = fda.alloc_prefill_workspace(128)
    want, wlse = ref.attention_blocks(f, q, 8, 128 ** -0.5)
    for kv in ("e4m3", "f16"):
        fda.fd_debug_set_wait_limit(3_000_000, True)
        try:
            if kv == "f16":
                g = ref.Filled(ref.Batch([200, 1], [10, 700], 2, 128, "f16", 16, seed=11), seed=11)
                _attend(fda, g, q, 8, ws)
            else:
                _attend(fda, f, q, 8, ws)
        finally:
            fda.fd_debug_set_wait_limit(0, False)
        assert fda.fd_check_device_error(ws)[0] == fda.FD_ERR_DEVICE_TIMEOUT
    out, lse = _attend(fda, f, q, 8, ws)
    _ok(fda, ws)
    _compare(f, out, lse, want, wlse, "f16")


@pytest.mark.parametrize("kv,scales", [("f16", "tensor"), ("e4m3", "tensor"), ("i8", "token")])
def test_attention_waits_that_run_out_in_the_middle(kv, scales):
    """Limits so short that waits run out with copies and products in flight:
    the call ends, reports it, and the next one is right."""
    fda = lib()
    bt = ref.Batch([300, 1, 64, 3], [40, 2000, 0, 900], 2, 128, kv, 64, seed=21)
    f = ref.Filled(bt, seed=21, scales=scales)
    q = _queries(bt, 8, "f16", 21)
    ws = fda.alloc_prefill_workspace(128)
    want, wlse = ref.attention_blocks(f, q, 8, 128 ** -0.5)
    for limit in (1, 100, 1000, 5000, 30000):
        fda.fd_debug_set_wait_limit(limit, False)
        try:
            for _ in range(4):
                _attend(fda, f, q, 8, ws)
                assert fda.fd_check_device_error(ws)[0] in (fda.FD_OK, fda.FD_ERR_DEVICE_TIMEOUT)
        finally:
            fda.fd_debug_set_wait_limit(0, False)
    out, lse = _attend(fda, f, q, 8, ws)
    _ok(fda, ws)
    _compare(f, out, lse, want, wlse, "f16")


# ---------------------------------------------------------------------------
# together, on streams, in graphs
# ---------------------------------------------------------------------------

def test_prompt_then_decode_then_read_back():
    """A prompt in two chunks (rotated, written, attended), then decode steps
    through the same cache, then the cache read back: each stage against a
    plain statement of the whole."""
    fda = lib()
    B, QH, KVH, D, P, rot = 3, 8, 2, 128, 16, 128
    chunks = [[50, 7, 130], [20, 1, 3]]
    steps = 3
    total = [sum(c) + steps for c in zip(*chunks)]
    g = torch.Generator().manual_seed(3)
    pages = [-(-t // P) for t in total]
    perm = torch.randperm(sum(pages) + 2, generator=g).int()
    bt = torch.zeros((B, max(pages)), dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        bt[b, :n] = perm[at:at + n]
        at += n
    kc, vc = (torch.zeros((sum(pages) + 2, P, KVH, D), dtype=torch.bfloat16, device=DEV)
              for _ in range(2))
    tab = fda.rotary_table(max(total), rot, theta=10000.0)
    host = torch.from_numpy(ref.table(max(total), rot, 10000.0))
    btd = bt.to(DEV)
    ws = fda.alloc_prefill_workspace(D)
    K = [torch.zeros((0, KVH, D), dtype=torch.float64) for _ in range(B)]
    V = [torch.zeros((0, KVH, D), dtype=torch.float64) for _ in range(B)]
    seq = [0] * B

    def turned(x, pos):   # rounded to bf16, as the cache and q_out are
        return ref.rotate(x, host, pos, rot, False, torch.float64).bfloat16().double()

    def expect(q, new):
        outs = []
        for b, n in enumerate(new):
            for j in range(n):
                i = sum(new[:b]) + j
                pos = torch.tensor([seq[b] - n + j])
                qq = turned(q[i:i + 1], pos)[0]
                k, v = K[b][:seq[b] - n + j + 1], V[b][:seq[b] - n + j + 1]
                k, v = (x.repeat_interleave(QH // KVH, 1) for x in (k, v))
                w = torch.softmax(torch.einsum("hd,thd->ht", qq, k) * D ** -0.5, -1)
                outs.append(torch.einsum("ht,thd->hd", w, v))
        return torch.stack(outs)

    def write(k, v, new):
        for b, n in enumerate(new):
            i = sum(new[:b])
            pos = torch.arange(seq[b], seq[b] + n)
            K[b] = torch.cat([K[b], turned(k[i:i + n], pos)])
            V[b] = torch.cat([V[b], v[i:i + n].double()])
            seq[b] += n

    for new in chunks + [[1] * B] * steps:
        n = sum(new)
        q, k, v = (torch.randn((n, h, D), generator=g).bfloat16() for h in (QH, KVH, KVH))
        pos = torch.tensor(seq, dtype=torch.int32, device=DEV)
        write(k, v, new)
        sl = torch.tensor(seq, dtype=torch.int32, device=DEV)
        qs = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
        if new != [1] * B:
            out, _ = fda.prefill_attention(q.to(DEV), kc, vc, qs, sl, block_table=btd,
                                           k_new=k.to(DEV), v_new=v.to(DEV), positions=pos,
                                           rotary=tab, workspace=ws)
        else:
            qt = fda.append_kv(k.to(DEV), v.to(DEV), kc, vc, qs, pos, q=q.to(DEV), rotary=tab,
                               block_table=btd, workspace=ws)
            out, _ = fda.decode_attention(qt, kc, vc, sl, block_table=btd)
        torch.cuda.synchronize()
        want = expect(q, new)
        # the cache and the queries may round the other way where fp32 and
        # 64-bit rotations straddle a tie: one bf16 step in rare elements
        assert float((out.double().cpu() - want).abs().max()) <= 3e-2
        assert float((out.double().cpu() - want).norm() / want.norm()) <= 2.0 ** -8
    ko, vo = fda.read_kv(kc, vc, torch.tensor(np.concatenate([[0], np.cumsum(seq)]),
                                              dtype=torch.int32, device=DEV), sum(seq),
                         block_table=btd, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(vo.double().cpu(), torch.cat(V))
    d = (ko.double().cpu() - torch.cat(K)).abs()
    assert torch.all(d <= 2.0 ** -7 * torch.cat(K).abs() + 2.0 ** -20)
    _ok(fda, ws)


def test_prompt_path_in_a_graph():
    """The prompt path captured once and replayed after queries, new rows and
    lengths change in place; a second graph shares the workspace."""
    fda = lib()
    bt = ref.Batch([60, 1, 20], [100, 300, 0], 2, 64, "e4m3", 16, seed=12)
    f = ref.Filled(bt, seed=12)
    kw, ix = f.device(DEV), bt.index(DEV)
    ws = fda.alloc_prefill_workspace(64)
    qs = torch.from_numpy(bt.q_start).to(DEV)
    sl = torch.tensor(bt.seq, dtype=torch.int32, device=DEV)
    bufs = [torch.zeros((bt.tokens, 8, 64), dtype=torch.float16, device=DEV) for _ in range(2)]
    graphs, outs = [], []
    for q in bufs:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            fda.prefill_attention(q, kw["k_cache"], kw["v_cache"], qs, sl, k_scale=kw["k_scale"],
                                  v_scale=kw["v_scale"], workspace=ws, **ix)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fda.prefill_attention(q, kw["k_cache"], kw["v_cache"], qs, sl,
                                              k_scale=kw["k_scale"], v_scale=kw["v_scale"],
                                              workspace=ws, **ix))
        graphs.append(g)
    for step in range(3):
        for i in (0, 1):
            q = _queries(bt, 8, "f16", 20 + 2 * step + i)
            bufs[i].copy_(q)
            if step == 2:   # shorter sequences: the last rows are new tokens again
                bt.seq = [140, 260, 20]
                sl.copy_(torch.tensor(bt.seq, dtype=torch.int32))
            graphs[i].replay()
            torch.cuda.synchronize()
            want, wlse = ref.attention_blocks(f, q, 8, 0.125)
            _compare(f, outs[i][0].double().cpu(), outs[i][1].double().cpu(), want, wlse, "f16")
    _ok(fda, ws)


def test_prompt_path_on_other_streams():
    """Two streams at once, each with its own workspace and inputs; a stream
    given by its handle."""
    fda = lib()
    cases = []
    for i in range(2):
        bt = ref.Batch([150, 1, 33], [0, 500, 7], 2, 128, "bf16", 16, seed=30 + i)
        f = ref.Filled(bt, seed=30 + i)
        q = _queries(bt, 8, "bf16", 30 + i)
        cases.append((bt, f, q, f.device(DEV), bt.index(DEV), torch.from_numpy(bt.q_start).to(DEV),
                      torch.tensor(bt.seq, dtype=torch.int32, device=DEV), q.to(DEV),
                      fda.alloc_prefill_workspace(128), torch.cuda.Stream()))
    torch.cuda.synchronize()
    res = []
    for rep in range(4):
        for i, (bt, f, q, kw, ix, qs, sl, qd, ws, st) in enumerate(cases):
            out = fda.prefill_attention(qd, kw["k_cache"], kw["v_cache"], qs, sl, workspace=ws,
                                        stream=st if rep % 2 else st.cuda_stream, **ix)
            res.append((i, out))
    # without a workspace of the caller's, on a stream of its own
    bt, f, q, kw, ix, qs, sl, qd, ws, st = cases[0]
    res.append((0, fda.prefill_attention(qd, kw["k_cache"], kw["v_cache"], qs, sl, stream=st, **ix)))
    torch.cuda.synchronize()
    for i, (out, lse) in res:
        bt, f, q = cases[i][:3]
        want, wlse = ref.attention_blocks(f, q, 8, 128 ** -0.5)
        _compare(f, out.double().cpu(), lse.double().cpu(), want, wlse, "bf16")


def test_prompt_path_from_several_threads():
    """Three host threads at once, each with its own stream, workspace, format
    and shape (descriptors, kernel variants and limits set for the first time
    by whoever comes first)."""
    fda = lib()
    jobs = []
    for i, (kv, x16, d, page, scales) in enumerate([("e4m3", "f16", 128, 64, "tensor"),
                                                    ("bf16", "bf16", 64, 0, "tensor"),
                                                    ("i8", "f16", 128, 16, "token")]):
        bt = ref.Batch([90 + 40 * i, 1, 17], [600, 33, 0], 2, d, kv, page, seed=70 + i)
        f = ref.Filled(bt, seed=70 + i, scales=scales)
        q = _queries(bt, 8, x16, 70 + i)
        kw = f.device(DEV)
        args = (q.to(DEV), kw.pop("k_cache"), kw.pop("v_cache"),
                torch.from_numpy(bt.q_start).to(DEV),
                torch.tensor(bt.seq, dtype=torch.int32, device=DEV))
        jobs.append((f, q, x16, args, {**kw, **bt.index(DEV)}, fda.alloc_prefill_workspace(d),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    res, wrong = [None] * len(jobs), []
    gate = threading.Barrier(len(jobs))

    def work(i):
        try:
            f, q, x16, args, kw, ws, st = jobs[i]
            gate.wait()
            for _ in range(25):
                table = fda.rotary_table(300 + i, 32, stream=st)
                res[i] = (*fda.prefill_attention(*args, workspace=ws, stream=st, **kw), table)
            st.synchronize()
        except Exception as e:      # noqa: BLE001 (shown by the assertion below)
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    torch.cuda.synchronize()
    for i, (f, q, x16, _, _, ws, _) in enumerate(jobs):
        _ok(fda, ws)
        out, lse, table = res[i]
        want, wlse = ref.attention_blocks(f, q, 8, f.batch.d ** -0.5)
        _compare(f, out.double().cpu(), lse.double().cpu(), want, wlse, x16)
        ang = ref.table(300 + i, 32, 10000.0)
        assert np.abs(table.double().cpu().numpy() - ang).max() <= 5 * 2.0 ** -24 + 300 * 2.0 ** -52


def test_prompt_path_far_into_a_large_cache():
    """Rows whose element offsets pass 32 bits (a 5 GB cache)."""
    fda = lib()
    rows, KVH, D = 5 * 10 ** 6, 8, 128
    kc, vc = (torch.zeros((rows, KVH, D), dtype=torch.uint8, device=DEV) for _ in range(2))
    start = rows - 300
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn((200, KVH, D), generator=g).half() for _ in range(2))
    q = torch.randn((200, 8, D), generator=g).half()
    i32 = dict(dtype=torch.int32, device=DEV)
    qs, sl = torch.tensor([0, 200], **i32), torch.tensor([200], **i32)
    first = torch.tensor([start], **i32)
    ws = fda.alloc_prefill_workspace(D)
    scale = 5.0 / 448
    out, lse = fda.prefill_attention(q.to(DEV), kc, vc, qs, sl, kv_start_idx=first,
                                     k_new=k.to(DEV), v_new=v.to(DEV),
                                     positions=torch.tensor([0], **i32), k_scale=scale,
                                     v_scale=scale, workspace=ws)
    ko, vo = fda.read_kv(kc, vc, qs, 200, kv_start_idx=first, k_scale=scale, v_scale=scale,
                         workspace=ws)
    torch.cuda.synchronize()
    _ok(fda, ws)
    assert int(kc[:start].count_nonzero()) == 0 and int(kc[start + 200:].count_nonzero()) == 0
    kd, vd = ko.double().cpu(), vo.double().cpu()
    assert float((kd - k.double()).abs().max()) <= 2.0 ** -4 * 5     # e4m3: half a step
    s = torch.einsum("ihd,thd->hit", q.double(), kd) * D ** -0.5
    s = s.masked_fill(torch.triu(torch.ones(200, 200, dtype=torch.bool), 1), -math.inf)
    want = torch.einsum("hit,thd->ihd", torch.softmax(s, -1), vd)
    assert float((out.double().cpu() - want).abs().max()) <= 2.0 ** -10 * 5.5 + 2.0 ** -10
