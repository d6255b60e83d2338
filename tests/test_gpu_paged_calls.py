"""Calls of the paged prefix-KV cache (include/mot_paged.h) around the kernels:
addresses that are no device memory of the current device."""
from ctypes import byref, c_void_p

import pytest
import torch

from mot_flow_matching_b200 import _abi
from tests.gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu


def test_create_refuses_gains_in_host_memory(cuda_ready):
    # on the host, before the kernels that would read them
    ensure_built()
    cfg = _abi.MotPagedConfig(4, 2, 128, 16, 0, 1e-6, 1e6, 64, 1, 8, 4)
    dev = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    host, pinned = torch.ones(128, dtype=torch.bfloat16), torch.ones(128, dtype=torch.bfloat16).pin_memory()
    for q, k in ((host, dev), (dev, host), (pinned, dev), (dev, pinned)):
        out = c_void_p(1)
        w = _abi.MotPagedWeights(q.data_ptr(), k.data_ptr())
        assert _abi.lib().mot_paged_create(byref(cfg), byref(w), None, byref(out)) == _abi.MOT_ERR_INVALID_ARGUMENT
        assert out.value is None
    w = _abi.MotPagedWeights(dev.data_ptr(), dev.data_ptr())
    out = c_void_p()
    assert _abi.lib().mot_paged_create(byref(cfg), byref(w), None, byref(out)) == _abi.MOT_OK
    _abi.lib().mot_paged_destroy(out)
