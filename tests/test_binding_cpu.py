"""The binding where there is no GPU: it imports, and refuses tensors in its own words."""
import os
import subprocess
import sys

import pytest
import torch

from block_sparse_top_summary_b200 import abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _calls():
    K, s = torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2)
    i = torch.zeros(1, dtype=torch.int32)
    yield "Kp", lambda: abi.ssa_decode_paged_q8(torch.zeros(1, 4, 64), K, s, K, s, None, i[None], i,
                                                16, 9)
    yield "Kp", lambda: abi.ssa_append_paged_q8(K, s, K, s, None, i, i, i, s, s, 16, max_blocks=1)
    yield "have", lambda: abi.ssa_page_plan(i, i, i[None], i, torch.zeros(2, dtype=torch.int32), 16,
                                            4)


def test_tensors_on_the_host_are_refused_with_or_without_a_driver():
    for name, call in _calls():
        with pytest.raises(ValueError, match=name + " must be a CUDA tensor"):
            call()


def test_import_and_refusals_on_a_torch_without_cuda():
    # what such a torch lacks is taken away before the package is imported
    code = """
import sys, torch
sys.path[:0] = [%r, %r]
for name in [n for n in dir(torch._C) if n.startswith("_cuda_get")]:
    delattr(torch._C, name)
torch.cuda.is_available = lambda: False
import block_sparse_top_summary_b200
import test_binding_cpu
test_binding_cpu.test_tensors_on_the_host_are_refused_with_or_without_a_driver()
""" % (ROOT, os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0, r.stderr
