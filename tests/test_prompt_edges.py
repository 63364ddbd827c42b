"""CPU checks of the prompt path's arguments at their edges: arrays without
rows, arrays that overlap, tables that are not on a GPU."""
import pytest
import torch

import flash_decoding_attention_gb300 as fda
from test_prompt_args import _append, _prefill, _read, c  # noqa: F401 (c: the library)

# Past the argument checks a host without a device answers FD_ERR_CUDA where the
# number of SMs is needed.
DONE = (fda.FD_OK, fda.FD_ERR_CUDA)


def test_packed_arrays_without_rows_may_be_null(c):  # noqa: F811
    assert _append(c, n=0, q=None, qo=None, kn=None, vn=None) == fda.FD_OK
    assert _append(c, n=0, kn=None, vn=None, qo=None) == fda.FD_OK
    assert _read(c, n=0, ko=None, vo=None) == fda.FD_OK
    assert _prefill(c, n=0, q=None, out=None, lse=None) in DONE
    # every other argument is looked at all the same
    assert _append(c, n=0, kn=None, vn=None, pos=None) == fda.FD_ERR_INVALID_ARG
    assert _append(c, n=0, kn=None, vn=None, d=96) == fda.FD_ERR_UNSUPPORTED
    assert _read(c, n=0, ko=None, vo=None, os=None) == fda.FD_ERR_INVALID_ARG
    assert _prefill(c, n=0, q=None, out=None, sl=None) == fda.FD_ERR_INVALID_ARG
    assert _prefill(c, n=0, q=None, out=None, qh=7) == fda.FD_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [
    dict(qo=0x100000 + 2048), dict(qo=0x100000 - 16),               # q, not in place
    dict(qst=9 * 128, qo=0x100000 + 9 * 9 * 256),                   # the last of strided tokens
    dict(qo=0x200000), dict(qo=0x200000 + 9 * 512 + 256), dict(qo=0x200000 - 10 * 2048 + 16),
    dict(qo=0x300000 + 512),
])
def test_turned_queries_may_not_overlap_what_is_read(c, over):  # noqa: F811
    """q_out is written by blocks while others still read q, k_new and v_new."""
    a = dict(q=0x100000, kn=0x200000, vn=0x300000, qo=0x400000)
    a.update(over)
    assert _append(c, **a) == fda.FD_ERR_INVALID_ARG


def test_rotary_table_is_made_on_a_gpu():
    with pytest.raises(ValueError, match="GPU"):
        fda.rotary_table(10, 16, out=torch.empty((10, 16)))
    with pytest.raises(ValueError, match="GPU"):
        fda.rotary_table(10, 16, out=torch.empty((10, 16)), stream=0)
    with pytest.raises(ValueError, match="GPU"):
        fda.rotary_table(10, 16, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        fda.rotary_table(10, 16, device="cpu", stream=0)
