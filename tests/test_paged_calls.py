"""CPU tests of the paged operators' calls: what is refused, and what is not, before anything reaches CUDA."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

from rotation_preconditioned_quantization_b200 import _lib, api, paged

EINVAL, EUNS, OK = _lib.OCTO_EINVAL, _lib.OCTO_EUNSUPPORTED, _lib.OCTO_OK


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


def _cpu(H=2, d=64, b=2, page=16, pages=4):
    lay = api.Layout(d, b)
    return lay, api.DeviceTables.build(lay, 0, H, device="cpu"), paged.PagedCache.empty(lay, pages, H, page, device="cpu")


def test_no_wait_of_the_paged_kernels_is_unbounded():
    """Roles that give up a bounded wait leave the others: within the roles nothing may wait without a limit, so no
    barrier of named threads, and every poll of an mbarrier is in the bounded loop."""
    src = os.path.join(os.path.dirname(paged.__file__), "csrc")
    for name in ("octo_paged.cuh", "octo_paged_attn.cu", "octo_paged_mass.cu"):
        text = open(os.path.join(src, name)).read()
        assert not re.search(r"\bbar(rier)?\.(sync|red)|named_sync", text), name
        assert len(re.findall(r"mbarrier\.(try|test)_wait", text)) == (1 if name == "octo_paged.cuh" else 0)
        roles = re.findall(r"__device__ __forceinline__ bool \w+_role\(.*?\n}\n", text, re.S)
        assert all("__syncthreads" not in r for r in roles)
    wait = open(os.path.join(src, "octo_paged.cuh")).read().split("bool bar_wait(")[1].split("\n}\n")[0]
    assert re.search(r"it < \(1 << \d+\)", wait) and "while" not in wait


@pytest.mark.parametrize("d", [64, 128])
def test_paged_scratch_lies_behind_the_words_that_decode_keeps(d):
    """octo_decode_attn's status word and the arrival counters of its at most 65535 cache heads come first."""
    lib, lay = _lib.lib(), api.Layout(d, 3)
    front = 256 + 4 * 65535
    assert lib.octo_paged_attn_workspace(lay.ref, 1, 1, 1, 1) >= front + 148 * 3 * 256 * d * 4
    assert lib.octo_paged_mass_workspace(lay.ref, 64, 1, 1, 1) >= front + 64 * d * 4
