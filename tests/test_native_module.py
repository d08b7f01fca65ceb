"""The binding's extension module belongs to one torch: another one gets its own build."""
import os
import subprocess

import torch

from quantized_gemm_rank_gb300 import build


def test_a_module_of_another_torch_is_not_taken(monkeypatch):
    mine = build.build_native()
    assert os.path.exists(mine)
    runs = []

    def compiler(cmd, **kw):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", compiler)
    assert build.build_native() == mine and not runs
    size = os.path.getsize(mine)
    monkeypatch.setattr(torch, "__version__", "0.0.1+test")
    other = build.build_native()
    try:
        assert len(runs) == 1 and other != mine and os.path.getsize(mine) == size
    finally:
        if other != mine:
            os.remove(other)
