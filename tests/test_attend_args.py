"""CPU checks of the page bookkeeping's call with the attention's lengths: it
refuses what the call without them refuses, and arrays of its own."""
import pytest

import flash_decoding_attention_gb300 as fda


@pytest.fixture(scope="module")
def c():
    from flash_decoding_attention_gb300 import build
    build.build()
    return fda.load_library()


def _call(c, **over):
    a = dict(bt=0x1000, stride=4, sl=0x2000, new=0x3000, free=0x4000, cap=100, count=0x5000, batch=2,
             page=16, win=4, sinks=1, rel=0xC000, slo=0x6000, co=0x7000, ro=0xD000, qs=0x8000,
             pos=0x9000, slots=0xA000, ns=10, att=0xE000, ws=0xB000, wsb=1 << 20)
    a.update(over)
    return c.fd_assign_pages_attended(
        a["bt"], a["stride"], a["sl"], a["new"], a["free"], a["cap"], a["count"], a["batch"],
        a["page"], a["win"], a["sinks"], a["rel"], a["slo"], a["co"], a["ro"], a["qs"], a["pos"],
        a["slots"], a["ns"], a["att"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,status", [
    (dict(att=0xE002), 1),                                          # not aligned
    (dict(att=0x2000), 1), (dict(att=0x3004), 1), (dict(att=0x1010), 1), (dict(att=0x8008), 1),
    (dict(att=0x9000), 1), (dict(att=0x6004), 1), (dict(att=0xD000), 1), (dict(att=0xA000), 1),
    (dict(att=0xB000), 1),                                          # on another array
    (dict(bt=None), 1), (dict(win=0, sinks=0), 1), (dict(page=24), 2), (dict(wsb=256), 3),
    (dict(att=None, ws=None), 1), (dict(att=None, qs=0x2000), 1),
])
def test_refusals(c, over, status):
    assert _call(c, **over) == status
