"""The binding of the adapters and the experts, where the process has passed no tensor before."""
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
