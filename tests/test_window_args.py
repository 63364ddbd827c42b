"""CPU checks of the windowed entry points' arguments: the C entries refuse bad
ones on the host (fake pointers are never dereferenced), the torch wrappers
refuse bad tensors."""
import pytest
import torch

import flash_decoding_attention_gb300 as fda


@pytest.fixture(scope="module")
def c():
    from flash_decoding_attention_gb300 import build
    build.build()
    return fda.load_library()


def _decode(c, **over):
    a = dict(q=0x1000, kn=None, vn=None, k=0x2000, v=0x3000, kv_start=0x4000, bt=None, bts=0,
             pos=None, sl=0x5000, rows=100, batch=2, qh=8, kvh=2, d=128, page=0, win=16, sinks=4,
             ss=0.1, ks=1.0, vs=1.0, kind=0, kss=None, vss=None, qdt=0, kvdt=0, out=0x6000,
             lse=0x7000, ws=0x8000, wsb=1 << 30)
    a.update(over)
    return c.fd_decode_attention_window(
        a["q"], a["kn"], a["vn"], a["k"], a["v"], a["kv_start"], a["bt"], a["bts"], a["pos"],
        a["sl"], a["rows"], a["batch"], a["qh"], a["kvh"], a["d"], a["page"], a["win"], a["sinks"],
        a["ss"], a["ks"], a["vs"], a["kind"], a["kss"], a["vss"], a["qdt"], a["kvdt"], a["out"],
        a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,status", [
    (dict(win=0), 1), (dict(win=-1), 1), (dict(sinks=-1), 1), (dict(q=None), 1), (dict(k=None), 1),
    (dict(sl=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(ws=0x8010), 1),
    (dict(kn=0x9000), 1), (dict(kn=0x9000, vn=0xA000), 1), (dict(pos=0x9000), 1),
    (dict(kn=0x9008, vn=0xA000, pos=0xB000), 1), (dict(kv_start=None), 1),
    (dict(kn=0x9000, vn=0xA000, pos=0xB000, kvdt=2, ks=0.0), 1),
    (dict(qh=7), 1), (dict(qh=258), 2), (dict(d=96), 2), (dict(kind=2, kss=0x9000, vss=0xA000), 2),
    (dict(bt=0x9000, kv_start=None, bts=4, page=24, rows=96), 2), (dict(ss=float("nan")), 1),
    (dict(qdt=0, kvdt=1), 2), (dict(batch=0), 1),
])
def test_decode_refusals(c, over, status):
    assert _decode(c, **over) == status


def _prefill(c, **over):
    a = dict(q=0x1000, qst=8 * 128, k=0x2000, v=0x3000, kv_start=0x4000, bt=None, bts=0, qs=0x5000,
             sl=0x6000, n=10, rows=100, batch=2, qh=8, kvh=2, d=128, page=0, win=16, sinks=4, ss=0.1,
             ks=1.0, vs=1.0, kind=0, kss=None, vss=None, qdt=0, kvdt=0, out=0x7000, lse=0x8000,
             ws=0x9000, wsb=1 << 30)
    a.update(over)
    return c.fd_prefill_attention_window(
        a["q"], a["qst"], a["k"], a["v"], a["kv_start"], a["bt"], a["bts"], a["qs"], a["sl"], a["n"],
        a["rows"], a["batch"], a["qh"], a["kvh"], a["d"], a["page"], a["win"], a["sinks"], a["ss"],
        a["ks"], a["vs"], a["kind"], a["kss"], a["vss"], a["qdt"], a["kvdt"], a["out"], a["lse"],
        a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,status", [
    (dict(win=0), 1), (dict(sinks=-1), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(sl=None), 1),
    (dict(qs=None), 1), (dict(ws=0x9080), 1), (dict(qst=8 * 128 + 2), 1), (dict(n=-1), 1),
    (dict(qh=7), 1), (dict(d=32), 2), (dict(kv_start=None), 1), (dict(rows=1 << 31), 2),
    (dict(out=0x1010), 1),
])
def test_prefill_refusals(c, over, status):
    assert _prefill(c, **over) == status


def test_wrapper_refusals():
    t = torch.zeros
    q = t(2, 8, 64, dtype=torch.float16)
    k = t(10, 2, 64, dtype=torch.float16)
    i = t(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="give window"):
        fda.decode_attention(q, k, k, i, kv_start_idx=i, sinks=4)
    with pytest.raises(ValueError, match="give window"):
        fda.prefill_attention(q, k, k, t(3, dtype=torch.int32), i, kv_start_idx=i, sinks=4)
    for bad in (dict(window=0), dict(window=-5), dict(window=3, sinks=-1),
                dict(window=(1 << 32) + 5), dict(window=3, sinks=1 << 32)):
        with pytest.raises(ValueError, match="window must be"):
            fda.decode_attention(q, k, k, i, kv_start_idx=i, **bad)
        with pytest.raises(ValueError, match="window must be"):
            fda.prefill_attention(q, k, k, t(3, dtype=torch.int32), i, kv_start_idx=i, **bad)
    with pytest.raises(ValueError, match="on a GPU"):
        fda.decode_attention(q, k, k, i, kv_start_idx=i, window=3)
