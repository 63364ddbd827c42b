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
