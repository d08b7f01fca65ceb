"""The workspace of an int8 product depends on its matrices and sizes alone: asked for where no device is visible, it is the
same."""
import json
import os
import random
import subprocess
import sys

import pytest
import torch

import quantized_gemm_rank_gb300 as mc2

ASK = """
import ctypes, json, sys
import quantized_gemm_rank_gb300 as mc2
n, sizes = ctypes.c_size_t(0), json.load(sys.stdin)
def ask(m, cols, k, nk):
    st = mc2.lib().mc2_quant_matmul_workspace(65536, k, 65536, k if nk else cols, nk, m, cols, k, None, 0, 65536, cols, ctypes.byref(n))
    return [st, n.value]
print(json.dumps([ask(*s) for s in sizes]))
"""


@pytest.mark.gpu
def test_the_same_without_a_device():
    rng = random.Random(1)
    sizes = [(int(2 ** rng.uniform(3, 11)), int(2 ** rng.uniform(6, 14)) // 16 * 16, int(2 ** rng.uniform(6, 14)) // 16 * 16, rng.random() < 0.7)
             for _ in range(4000)]
    torch.zeros(1, device="cuda")
    root = os.path.dirname(os.path.dirname(os.path.abspath(mc2.__file__)))

    def answers(**env):
        return json.loads(subprocess.run([sys.executable, "-c", ASK], input=json.dumps(sizes), capture_output=True, text=True, check=True,
                                         cwd=root, env={**os.environ, **env}).stdout)

    here, there = answers(), answers(CUDA_VISIBLE_DEVICES="")
    differ = [(s, a, b) for s, a, b in zip(sizes, here, there) if a != b]
    assert not differ, f"{len(differ)} of {len(sizes)} sizes, first {differ[0]}"
    assert {a[1] > 0 for a in here} == {True, False} and all(a[0] == mc2.MC2_OK for a in here)
