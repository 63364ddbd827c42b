"""GPU tests of the normed append's sum of squares next to the middle of two fp32
numbers."""
import numpy as np
import pytest
import torch

from gpu_util import lib
from test_gpu_norms import DEV

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt,small,times", [(torch.float16, 2.0 ** -24, 1),
                                            (torch.bfloat16, 2.0 ** -25, 24),
                                            (torch.float16, 2.0 ** -18, 1)])
def test_a_sum_next_to_the_middle_of_two_numbers(dt, small, times, d):
    """1 + 2^-24 and a little: the sum is one of its neighbours 1 and 1 + 2^-23,
    whatever the places of the elements, and the upper one where the little is
    more than 2^-40.  A scale per token of an INT8 cache tells which: the largest
    element is 1, so it is the head's factor by 127.  (Everything twice with 64
    elements: square roots of odd powers of two tell neighbours apart.)"""
    fda = lib()
    n, m = 300, 128 // d
    g = torch.Generator().manual_seed(d)
    k = torch.zeros((n, 1, d), dtype=dt)
    for i in range(n):
        at = torch.randperm(d, generator=g)
        k[i, 0, at[:m]] = 1.0
        k[i, 0, at[m:2 * m]] = 2.0 ** -12
        k[i, 0, at[2 * m:(2 + times) * m]] = small
    little = times * small ** 2
    exact = k.double().square().sum(-1)
    assert torch.all(exact == m * (1 + 2.0 ** -24 + little))
    kc, vc = (torch.zeros((n, 1, d), dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((n, 1), device=DEV) for _ in range(2))
    eps = 1e-30                     # nothing beside the sum
    fda.append_kv(k.to(DEV), k.to(DEV), kc, vc, torch.tensor([0, n], **I32), torch.zeros(1, **I32),
                  kv_start_idx=torch.zeros(1, **I32), k_scales=ks, v_scales=vs,
                  k_norm=torch.ones(d, device=DEV), norm_eps=eps)
    torch.cuda.synchronize()
    f32 = np.float32
    either = []
    for s in (f32(1), np.nextafter(f32(1), f32(2))):
        either.append(float(f32(1) / np.sqrt(f32(m * s * f32(1 / d)) + f32(eps)) / f32(127)))
    assert either[0] != either[1]
    got = ks.cpu().view(-1).tolist()
    assert set(got) <= set(either), set(got)
    if little > 2.0 ** -40:
        assert set(got) == {either[1]}
