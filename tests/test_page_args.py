"""CPU checks of the page bookkeeping's arguments, and of its plain statement."""
import pytest
import torch

import flash_decoding_attention_gb300 as fda
import pages_ref


@pytest.fixture(scope="module")
def c():
    from flash_decoding_attention_gb300 import build
    build.build()
    return fda.load_library()


def _call(c, **over):
    a = dict(bt=0x1000, stride=4, sl=0x2000, new=0x3000, free=0x4000, cap=100, count=0x5000, batch=2,
             page=16, win=0, sinks=0, rel=None, slo=0x6000, co=0x7000, ro=None, qs=0x8000,
             pos=0x9000, slots=0xA000, ns=10, ws=0xB000, wsb=1 << 20)
    a.update(over)
    return c.fd_assign_pages(a["bt"], a["stride"], a["sl"], a["new"], a["free"], a["cap"], a["count"],
                             a["batch"], a["page"], a["win"], a["sinks"], a["rel"], a["slo"],
                             a["co"], a["ro"], a["qs"], a["pos"], a["slots"], a["ns"], a["ws"],
                             a["wsb"], None)


@pytest.mark.parametrize("over,status", [
    (dict(bt=None), 1), (dict(sl=None), 1), (dict(new=None), 1), (dict(free=None), 1),
    (dict(count=None), 1), (dict(slo=None), 1), (dict(co=None), 1), (dict(qs=None), 1),
    (dict(pos=None), 1), (dict(ws=None), 1), (dict(ws=0xB010), 1), (dict(wsb=256), 3),
    (dict(batch=0), 1), (dict(batch=(1 << 24) + 1), 1), (dict(stride=0), 1), (dict(cap=0), 1),
    (dict(cap=1 << 31), 1), (dict(page=0), 2), (dict(page=24), 2), (dict(page=512), 2),
    (dict(batch=1 << 20, stride=1 << 11, wsb=1 << 40), 2),
    (dict(win=-1), 1), (dict(sinks=4), 1), (dict(sinks=-1, win=4, rel=0xC000, ro=0xD000), 1),
    (dict(win=4), 1), (dict(win=4, rel=0xC000), 1), (dict(rel=0xC000, ro=0xD000), 1),
    (dict(ns=-1), 1), (dict(slots=None), 1), (dict(slots=0xA004), 1), (dict(bt=0x1002), 1),
    (dict(win=4, rel=0xC001, ro=0xD000), 1), (dict(ns=1 << 31), 1),
])
def test_refusals(c, over, status):
    assert _call(c, **over) == status


WIN = dict(win=4, sinks=1, rel=0xC000, ro=0xD000)


@pytest.mark.parametrize("over", [
    dict(qs=0x2000), dict(qs=0x2004), dict(pos=0x8008), dict(pos=0x3000), dict(slo=0x3000),
    dict(slo=0x2004), dict(slo=0x6000, pos=0x6004), dict(co=0x2000), dict(co=0x3004),
    dict(slots=0x8000), dict(slots=0x1000 - 8), dict(free=0x101C), dict(free=0x9000 - 396),
    dict(bt=0x4000), dict(ws=0x8000, qs=0x8400), dict(count=0x418C), dict(co=0x418C),
    dict(WIN, ro=0x2000), dict(WIN, ro=0xC004), dict(WIN, slo=0xC000), dict(WIN, qs=0xD004),
])
def test_arrays_lie_apart(c, over):
    """Two written arrays, or a written and a read one, that share an element."""
    assert _call(c, **over) == 1


def test_workspace_bytes(c):
    assert c.fd_assign_pages_workspace_bytes(0) == 0
    assert c.fd_assign_pages_workspace_bytes((1 << 24) + 1) == 0
    assert c.fd_assign_pages_workspace_bytes(1000) >= 256 + 28 * 1000


def test_wrapper_refusals():
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="on a GPU"):
        fda.assign_pages(torch.zeros((2, 4), dtype=torch.int32), i, i, i, i[:1], 16)


def test_the_plain_statement():
    """A worked example: pages of four tokens, a window of six, one first token."""
    table = [[5, 6, 7, -9], [2, -9, -9, -9], [-9, -9, -9, -9]]
    free = [0, 1, 3, -7, -7, -7, -7, -7]
    got = pages_ref.step(table, [12, 3, 0], [1, -1, 5], free, 3, 4, 6, 1, [0, 0, 0], 8)
    q_start, positions, seq, count, released, slots, errors = got
    # token 12 sees 7 .. 12 and 0: columns 0 (first token) and 1 (token 7) stay
    assert q_start == [0, 1, 1, 6] and positions == [12, -1, 0] and seq == [13, 0, 5]
    # sequence 1's page 2 returns: stack 0 1 3 2; 2 to sequence 0, 3 and 1 to sequence 2
    assert table == [[5, 6, 7, 2], [2, -9, -9, -9], [3, 1, -9, -9]]
    assert count == 1 and free[:4] == [0, 1, 3, 2] and released == [1, 0, 1] and not errors
    assert slots == [2 * 4 + 0, 12, 13, 14, 15, 4, -1, -1]
    got = pages_ref.step(table, [15, 0, 5], [2, 0, 0], free, 1, 4, 6, 1, [1, 0, 1], None)
    # token 15 sees 10 .. 15: column 1 (tokens 4 .. 7) returns and is handed out again
    assert got[4] == [2, 1, 1] and got[1] == [-1, 0, 5] and got[6] == [5]
