"""CPU checks of the arguments of the packed append with norms and axes."""
import pytest
import torch

import flash_decoding_attention_gb300 as fda


@pytest.fixture(scope="module")
def c():
    from flash_decoding_attention_gb300 import build
    build.build()
    return fda.load_library()


def _append(c, **over):
    a = dict(q=0x1000000, qst=8 * 128, qo=0x2000000, kn=0x3000000, vn=0x4000000, kst=2 * 128,
             k=0x5000, v=0x6000, kv_start=0x7000, bt=None, bts=0, qs=0x8000, pos=0x9000, n=10,
             rows=100, batch=2, qh=8, kvh=2, d=128, page=0, rot=0xA000, rotp=64, rd=128, inter=0,
             qn=0xF000, kn_w=0xF100, f32=0, eps=1e-6, ap=0xF200, axes=3, ast=10,
             pa=bytes(i % 3 for i in range(64)), ks=1.0, vs=1.0, kind=0, kss=None, vss=None, ndt=0,
             kvdt=2, ws=0xB000, wsb=256)
    a.update(over)
    return c.fd_append_kv_normed(
        a["q"], a["qst"], a["qo"], a["kn"], a["vn"], a["kst"], a["k"], a["v"], a["kv_start"], a["bt"],
        a["bts"], a["qs"], a["pos"], a["n"], a["rows"], a["batch"], a["qh"], a["kvh"], a["d"],
        a["page"], a["rot"], a["rotp"], a["rd"], a["inter"], a["qn"], a["kn_w"], a["f32"], a["eps"],
        a["ap"], a["axes"], a["ast"], a["pa"], a["ks"], a["vs"], a["kind"], a["kss"], a["vss"],
        a["ndt"], a["kvdt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,status", [
    (dict(q=None), 1),                                  # q_norm without q
    (dict(qn=0xF001), 1), (dict(kn_w=0xF101), 1), (dict(qn=0xF002, f32=1), 1),
    (dict(eps=0.0), 1), (dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(axes=-1), 2), (dict(axes=5), 2), (dict(rot=None), 1), (dict(ap=None), 1),
    (dict(ap=0xF202), 1), (dict(pa=None), 1), (dict(ast=9), 1), (dict(ast=1 << 31), 1),
    (dict(pa=bytes([0] * 63 + [3])), 1), (dict(axes=1), 1),
    (dict(kn=None), 1), (dict(rd=24), 2), (dict(ks=0.0), 1), (dict(d=96), 2), (dict(wsb=128), 3),
])
def test_refusals(c, over, status):
    assert _append(c, **over) == status


def test_nothing_to_do_is_ok(c):
    assert _append(c, n=0) == 0
    assert _append(c, n=0, ap=None, ast=0) == 0
    # (a tensor of no tokens has no address)
    assert _append(c, n=0, q=None, qo=None, kn=None, vn=None, ap=None, ast=0) == 0


def test_wrapper_refusals():
    """The checks of norms and axes by themselves (the caches are on a GPU)."""
    q, k = torch.zeros(5, 4, 64).half(), torch.zeros(5, 2, 64).half()
    w, tab = torch.ones(64).half(), torch.zeros(9, 32)
    ap = torch.zeros((2, 5), dtype=torch.int32)

    def check(q=q, rotary=tab, q_norm=w, k_norm=w, axis_positions=None, pair_axes=None):
        return fda._norms_and_axes(q, k, 64, -1, rotary, q_norm, k_norm, axis_positions, pair_axes)

    assert check() == (False, b"")
    assert check(q_norm=w.float(), k_norm=None) == (True, b"")
    assert check(axis_positions=ap, pair_axes=[0, 1] * 8)[1] == bytes([0, 1] * 8)
    for bad in (dict(q=None), dict(q_norm=w[:32]), dict(q_norm=w.bfloat16()),
                dict(k_norm=w.float()), dict(q_norm=torch.ones(128).half()[::2]),
                dict(axis_positions=ap), dict(pair_axes=[0] * 16),
                dict(axis_positions=ap, pair_axes=[0] * 16, rotary=None),
                dict(axis_positions=ap, pair_axes=[0] * 15),
                dict(axis_positions=ap, pair_axes=[2] * 16),
                dict(axis_positions=ap, pair_axes=[-1] * 16),
                dict(axis_positions=ap.long(), pair_axes=[0] * 16),
                dict(axis_positions=ap[:, :4], pair_axes=[0] * 16),
                dict(axis_positions=ap[0], pair_axes=[0] * 16),
                dict(axis_positions=ap[:1].expand(2, 5), pair_axes=[0] * 16)):
        with pytest.raises(ValueError):
            check(**bad)
    with pytest.raises(TypeError):
        check(axis_positions=ap, pair_axes=16)
