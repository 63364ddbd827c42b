"""GPU tests of the normed append's signs: elements of both signs at the ends of
the range in one head."""
import pytest
import torch

from gpu_util import lib
from test_gpu_norms import DEV, EPS, normed

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dt,top,low", [(torch.float16, 65504.0, 2.0 ** -24),
                                        (torch.bfloat16, 1e18, 1e-30),
                                        (torch.bfloat16, 3e38, 1e-38)])
def test_signs_at_the_ends_of_the_range(dt, top, low):
    """Large and small elements of both signs in one head keep their signs."""
    fda = lib()
    q = torch.zeros((4, 1, 64), dtype=dt)
    q[0, 0, ::2], q[0, 0, 1::2] = top, -low
    q[1, 0, ::2], q[1, 0, 1::2] = -top, low
    q[2, 0, ::2], q[2, 0, 1::2] = low, -low
    q[3, 0, ::3], q[3, 0, 1::3] = -1.0, 1.5
    kc, vc = (torch.zeros((4, 1, 64), dtype=dt, device=DEV) for _ in range(2))
    w = torch.ones(64, device=DEV)
    got = fda.append_kv(q.to(DEV), q.to(DEV), kc, vc, torch.tensor([0, 4], **I32),
                        torch.zeros(1, **I32), q=q.to(DEV), q_norm=w, k_norm=w,
                        kv_start_idx=torch.zeros(1, **I32)).cpu()
    want = normed(q.float(), torch.ones(64), EPS)
    if top > 1e30:   # squares past fp32's range: an infinite sum
        want[:2] = 0
    want = want.to(dt)
    assert not torch.any(torch.isnan(got)) and not torch.any(torch.isnan(want))
    assert torch.equal(got, want) and torch.equal(kc.cpu(), want)
    big = want != 0
    assert big.any() and torch.equal(torch.signbit(got)[big], torch.signbit(q)[big])
