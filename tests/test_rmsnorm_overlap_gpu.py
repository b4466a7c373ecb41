"""A residual block's calls one after the other, each on what the ones before wrote, in the same
buffers and one workspace: the same bits with the programmatic overlap of consecutive kernels
(the default) and without it (FR_PDL=0, read once per process)."""
import os
import subprocess
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

CHILD = r'''
import sys, numpy as np, torch
sys.path.insert(0, sys.argv[1])
import reduction_pointwise_row_gb300 as fr
out = {}
gen = torch.Generator().manual_seed(5)
for rows, cols in ((1, 8192), (37, 1003), (3000, 96), (600, 4096), (310, 4097), (5, 20000)):
    x, r = (torch.randn(rows, cols, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    gamma = (1 + 0.1 * torch.randn(cols, generator=gen)).cuda()
    n = torch.tensor([rows, cols], device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    q = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
    ws = torch.empty(max(fr.fr_workspace_size("rmsnorm_backward", rows, cols, "bf16"), 1), dtype=torch.uint8,
                     device="cuda")
    dgamma, total = torch.empty_like(gamma), torch.zeros_like(gamma)
    for step in range(8):
        for site in range(3):
            fr.fr_rmsnorm(x, gamma, residual=r, p=0.1, rng=n, site=site, h=r, out=y, rstd=rstd)
            fr.fr_rmsnorm_backward(y, r, gamma, rstd, dh=x, p=0.1, rng=n, site=site, dx=x,
                                   want_dresidual=False, dgamma=dgamma, workspace=ws)
            fr.fr_rmsnorm_quant(x, gamma, residual=y, h=y, out=q, scale="group" if site else "row")
            fr.fr_dropout(y, 0.2, n, site, out=x)
            total += dgamma
        n[1] += 3
    for k, v in (("x", x), ("r", r), ("y", y), ("q", q)):
        out[f"{k}{rows}x{cols}"] = v.view(torch.uint8).cpu().numpy()
    out[f"dgamma{rows}x{cols}"] = total.cpu().numpy()
    assert total.isfinite().all() and x.isfinite().all()
np.savez(sys.argv[2], **out)
'''


def run_child(path, pdl: str):
    env = dict(os.environ, FR_PDL=pdl)
    subprocess.run([sys.executable, "-c", CHILD, ROOT, str(path)], env=env, check=True, timeout=600)
    return np.load(path)


def test_same_bits_with_and_without_the_overlap(tmp_path):
    on = run_child(tmp_path / "on.npz", "1")
    off = run_child(tmp_path / "off.npz", "0")
    assert set(on.files) == set(off.files)
    for k in on.files:
        assert on[k].tobytes() == off[k].tobytes(), k
