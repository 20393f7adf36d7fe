"""The binding of the adapters and the experts, where the process has passed no tensor before."""
import ctypes
import os
import subprocess
import sys

import pytest

import int4_weight_only_group_gb300 as kmr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FRESH = """
import torch
import int4_weight_only_group_gb300 as kmr
wide, ids = torch.zeros((4, 96)), torch.zeros(4, dtype=torch.int32)
try:
    kmr.kmr_lora_apply(0, wide[:, :64], wide[:, 64:], wide[:, 64:], 0, ids, 4, 96, 96)
except kmr.KmrError as e:
    print("library", e.code)
"""


def test_strided_rows_in_the_first_call_of_a_process():
    """Rows of wider matrices are taken whether or not a tensor was passed before (here to an adapter set given by its address: none)."""
    pytest.importorskip("torch")
    if not os.path.exists(kmr.library_path()):
        from int4_weight_only_group_gb300.build import build
        build()
    r = subprocess.run([sys.executable, "-c", FRESH], capture_output=True, text=True, cwd=ROOT)
    assert r.stdout.split() == ["library", str(kmr.KMR_ERR_INVALID_ARG)], r.stderr[-500:]


@pytest.mark.parametrize("kw,code", [(dict(inputs=(1 << 28) + 16), -2), (dict(outputs=(1 << 28) + 16), -2), (dict(outputs=1 << 29), -2),
                                     (dict(inputs=(1 << 31) - 16), -2), (dict(outputs=(1 << 31) - 16), -2)])
def test_adapters_whose_rows_pass_32_bits(kw, code):
    """A row's byte offsets are 32-bit numbers in the kernel: longer rows are refused (before any CUDA call)."""
    shape = dict(a=16, b=16, ranks=None, scales=None, adapters=1, inputs=64, outputs=32, max_rank=16)
    lora = kmr.LoraStruct(**{**shape, **kw})
    assert kmr.lib().kmr_lora_apply(ctypes.addressof(lora), 16, 16, 16, kmr.KMR_F32, 16, 1, 1 << 32, 1 << 32, None) == code
