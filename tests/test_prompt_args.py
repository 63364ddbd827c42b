"""CPU checks of the prompt path's arguments: the C entry points refuse bad
ones on the host, before any device work (fake pointers are never
dereferenced), and the torch wrappers refuse bad tensors."""
import os
import re

import pytest
import torch

import flash_decoding_attention_gb300 as fda


@pytest.fixture(scope="module")
def c():
    from flash_decoding_attention_gb300 import build
    build.build()
    return fda.load_library()


def _table(c, **over):
    a = dict(table=0x1000, positions=100, rot=64, theta=1e4, scaling=0, factor=1.0, original=8192.0,
             low=1.0, high=32.0, amplitude=1.0)
    a.update(over)
    return c.fd_rotary_table(a["table"], a["positions"], a["rot"], a["theta"], a["scaling"],
                             a["factor"], a["original"], a["low"], a["high"], a["amplitude"], None)


@pytest.mark.parametrize("over,status", [
    (dict(table=None), 1), (dict(table=0x1004), 1), (dict(positions=0), 1),
    (dict(positions=1 << 31), 1), (dict(rot=0), 2), (dict(rot=24), 2), (dict(rot=144), 2),
    (dict(theta=1.0), 1), (dict(theta=float("nan")), 1), (dict(theta=float("inf")), 1),
    (dict(scaling=3), 1), (dict(scaling=1, factor=0.5), 1), (dict(scaling=1, factor=float("nan")), 1),
    (dict(scaling=2, original=0.0), 1), (dict(scaling=2, low=2.0, high=2.0), 1),
    (dict(scaling=2, low=-1.0), 1), (dict(scaling=2, high=float("inf")), 1),
    (dict(amplitude=float("inf")), 1),
])
def test_rotary_table_refusals(c, over, status):
    assert _table(c, **over) == status


def _append(c, **over):
    a = dict(q=0x1000, qst=8 * 128, qo=0x2000, kn=0x3000, vn=0x4000, kst=2 * 128, k=0x5000, v=0x6000,
             kv_start=0x7000, bt=None, bts=0, qs=0x8000, pos=0x9000, n=10, rows=100, batch=2, qh=8,
             kvh=2, d=128, page=0, rot=0xA000, rotp=64, rd=128, inter=0, ks=1.0, vs=1.0, kind=0,
             kss=None, vss=None, ndt=0, kvdt=2, ws=0xB000, wsb=256)
    a.update(over)
    return c.fd_append_kv_packed(
        a["q"], a["qst"], a["qo"], a["kn"], a["vn"], a["kst"], a["k"], a["v"], a["kv_start"], a["bt"],
        a["bts"], a["qs"], a["pos"], a["n"], a["rows"], a["batch"], a["qh"], a["kvh"], a["d"],
        a["page"], a["rot"], a["rotp"], a["rd"], a["inter"], a["ks"], a["vs"], a["kind"], a["kss"],
        a["vss"], a["ndt"], a["kvdt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,status", [
    (dict(kn=None), 1), (dict(vn=None), 1), (dict(k=None), 1), (dict(qs=None), 1),
    (dict(pos=None), 1), (dict(ws=None), 1), (dict(ws=0xB010), 1), (dict(wsb=128), 3),
    (dict(qo=None), 1), (dict(q=0x1008), 1), (dict(qo=0x2004), 1), (dict(kn=0x3002), 1),
    (dict(qst=8 * 128 - 8), 1), (dict(qst=8 * 128 + 4), 1), (dict(kst=2 * 128 - 8), 1),
    (dict(kst=1 << 33), 1), (dict(q=0x2000, qst=9 * 128), 1),       # in place, but apart
    (dict(kv_start=None), 1), (dict(bt=0xC000, bts=4, page=16), 1),
    (dict(kv_start=None, bt=0xC000, bts=4, page=48, rows=96), 2),
    (dict(kv_start=None, bt=0xC000, bts=0, page=16, rows=96), 1),
    (dict(kv_start=None, bt=0xC000, bts=4, page=16, rows=100), 1),
    (dict(n=-1), 1), (dict(n=1 << 31), 1), (dict(batch=0), 1), (dict(qh=0), 1), (dict(kvh=0), 1),
    (dict(d=96), 2), (dict(rd=24), 2), (dict(rd=144), 2), (dict(d=64, rd=128), 2),
    (dict(rot=0xA004), 1), (dict(rotp=0), 1), (dict(ks=0.0), 1), (dict(vs=float("nan")), 1),
    (dict(kind=7), 1), (dict(kind=1), 1), (dict(kind=2, kss=0xD000, vss=0xE000, kvdt=0), 2),
    (dict(ndt=2), 1), (dict(kvdt=9), 1), (dict(ndt=0, kvdt=1), 2),
])
def test_append_packed_refusals(c, over, status):
    assert _append(c, **over) == status


def test_append_packed_of_nothing_is_ok(c):
    assert _append(c, n=0) == 0


def _read(c, **over):
    a = dict(k=0x1000, v=0x2000, kv_start=0x3000, bt=None, bts=0, os=0x4000, first=0x5000, n=10,
             rows=100, batch=2, kvh=2, d=128, page=0, ks=1.0, vs=1.0, kind=0, kss=None, vss=None,
             kvdt=2, odt=0, ko=0x6000, vo=0x7000, ws=0x8000, wsb=256)
    a.update(over)
    return c.fd_read_kv(a["k"], a["v"], a["kv_start"], a["bt"], a["bts"], a["os"], a["first"], a["n"],
                        a["rows"], a["batch"], a["kvh"], a["d"], a["page"], a["ks"], a["vs"],
                        a["kind"], a["kss"], a["vss"], a["kvdt"], a["odt"], a["ko"], a["vo"],
                        a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,status", [
    (dict(k=None), 1), (dict(os=None), 1), (dict(ko=None), 1), (dict(vo=0x7004), 1),
    (dict(first=0x5001), 1), (dict(n=-2), 1), (dict(batch=0), 1), (dict(d=32), 2),
    (dict(odt=2), 1), (dict(kvdt=0, odt=1), 2), (dict(kind=2, kss=0x9000), 1),
    (dict(ks=float("inf")), 1), (dict(wsb=0), 3), (dict(kv_start=None), 1),
])
def test_read_refusals(c, over, status):
    assert _read(c, **over) == status


def _prefill(c, **over):
    a = dict(q=0x1000, qst=8 * 128, k=0x2000, v=0x3000, kv_start=0x4000, bt=None, bts=0, qs=0x5000,
             sl=0x6000, n=10, rows=100, batch=2, qh=8, kvh=2, d=128, page=0, ss=0.1, ks=1.0, vs=1.0,
             kind=0, kss=None, vss=None, qdt=0, kvdt=0, out=0x7000, lse=0x8000, ws=0x9000,
             wsb=1 << 30)
    a.update(over)
    return c.fd_prefill_attention(
        a["q"], a["qst"], a["k"], a["v"], a["kv_start"], a["bt"], a["bts"], a["qs"], a["sl"], a["n"],
        a["rows"], a["batch"], a["qh"], a["kvh"], a["d"], a["page"], a["ss"], a["ks"], a["vs"],
        a["kind"], a["kss"], a["vss"], a["qdt"], a["kvdt"], a["out"], a["lse"], a["ws"], a["wsb"],
        None)


@pytest.mark.parametrize("over,status", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(sl=None), 1), (dict(qs=None), 1),
    (dict(ws=None), 1), (dict(ws=0x9080), 1), (dict(q=0x1008), 1), (dict(out=0x7008), 1),
    (dict(lse=0x8001), 1), (dict(qst=8 * 128 - 8), 1), (dict(qst=8 * 128 + 2), 1),
    (dict(n=-1), 1), (dict(qh=7), 1), (dict(qh=0), 1), (dict(qh=258, qst=258 * 128), 2),
    (dict(qh=4098, kvh=2049, qst=4098 * 128), 2),
    (dict(d=96), 2), (dict(rows=1 << 31), 2), (dict(rows=0), 1), (dict(ss=float("nan")), 1),
    (dict(kv_start=None), 1), (dict(qdt=3), 1), (dict(qdt=1), 2),
    (dict(kind=1, kss=0xA000, vss=0xB000), 2), (dict(kind=2, kvdt=3, kss=0xA002, vss=0xB000), 1),
    (dict(kv_start=None, bt=0xC000, bts=4, page=512, rows=1024), 2),
    (dict(out=0x1000), 1), (dict(out=0x5ff0), 1), (dict(q=0x7000 + 10 * 2048 - 16), 1),   # overlaps
])
def test_prefill_refusals(c, over, status):
    assert _prefill(c, **over) == status


def test_binding_has_the_headers_rotary_values():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                        "fd_attention.h")
    with open(path) as f:
        values = dict(re.findall(r"(FD_ROTARY_\w+) = (\d+)", f.read()))
    assert len(values) == 3 and set(int(x) for x in values.values()) == \
        set(fda.ROTARY_SCALINGS.values())
    for name, x in values.items():
        assert getattr(fda, name) == int(x)


def test_prefill_workspace_of_a_bad_head_dim(c):
    assert c.fd_prefill_workspace_bytes(96) == 0


def test_wrappers_refuse_bad_tensors():
    k = torch.zeros((100, 2, 64), dtype=torch.float16)
    i = torch.zeros(3, dtype=torch.int32)
    q = torch.zeros((4, 4, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="kv_start_idx"):
        fda.prefill_attention(q, k, k, i, i[:2])
    with pytest.raises(ValueError, match="kv_start_idx"):
        fda.read_kv(k, k, i, 4, kv_start_idx=i[:2], block_table=i.view(1, 3))
    with pytest.raises(ValueError, match="alike"):
        fda.read_kv(k, k[:50], i, 4, kv_start_idx=i[:2])
    with pytest.raises(ValueError, match="contiguous"):
        fda.read_kv(k[:, :, ::2], k[:, :, ::2], i, 4, kv_start_idx=i[:2])
    with pytest.raises(ValueError, match="GPU"):
        fda.append_kv(q[:, :2], q[:, :2], k, k, i, i[:2], kv_start_idx=i[:2])
    with pytest.raises(ValueError, match="scaling"):
        fda.rotary_table(10, 16, scaling="other", device="cpu")
    with pytest.raises(ValueError, match="dense"):
        fda._heads_rows("q", q.transpose(0, 1).contiguous().transpose(0, 1), 4, 64)
    with pytest.raises(ValueError, match="must be"):
        fda._heads_rows("q", q, 2, 64)
    assert fda._heads_rows("q", q[:, 1:3], 2, 64) == 4 * 64
    assert fda._heads_rows("q", q[:0], 4, 64) == 4 * 64
    with pytest.raises(ValueError, match="int32"):
        fda._index("seq_len", i.long(), 3, -1)
    with pytest.raises(ValueError, match="caches on"):
        fda._index("seq_len", i, 3, 0)
    with pytest.raises(ValueError, match="or neither"):
        fda._scale_kind(k.float(), None, 100, 2, -1)
    with pytest.raises(ValueError, match="dense fp32"):
        fda._scale_kind(torch.ones(3), torch.ones(3), 100, 2, -1)
    assert fda._scale_kind(torch.ones(2), torch.ones(2), 100, 2, -1) == fda.FD_SCALE_HEAD
    assert fda._scale_kind(torch.ones(100, 2), torch.ones(100, 2), 100, 2, -1) == fda.FD_SCALE_TOKEN
