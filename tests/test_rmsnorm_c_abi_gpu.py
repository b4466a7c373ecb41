"""A residual block's row operators from a plain C program (tests/c_abi/block_from_c.c,
built with gcc against include/fr.h): no Python or PyTorch in that process.  Its
outputs must meet the same bounds as the binding's."""
import subprocess

import numpy as np
import pytest
import torch

import rmsnorm_ref as ref
from test_c_abi_gpu import build_c_program
from test_rmsnorm_gpu import EPS, check_backward, check_norm, rng_of, values, vector

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def c_block(tmp_path_factory):
    return build_c_program("block_from_c", tmp_path_factory)


@pytest.mark.parametrize("rows,cols", [(200, 4096), (37, 1001), (3, 17000)])
def test_block_from_a_c_program(c_block, tmp_path, rows, cols):
    x, r, dy = (values(rows, cols, "bf16", 200 + i) for i in range(3))
    gamma, n = vector(cols, 20), rng_of(20)
    for name, v in (("x", x.view(torch.int16)), ("r", r.view(torch.int16)), ("dy", dy.view(torch.int16)),
                    ("gamma", gamma), ("rng", n)):
        v.numpy().tofile(str(tmp_path / f"{name}.bin"))
    p = subprocess.run([c_block, str(rows), str(cols), str(tmp_path)], capture_output=True, text=True,
                       timeout=120)
    assert p.returncode == 0, p.stderr

    def out(name, dtype):
        v = torch.from_numpy(np.fromfile(str(tmp_path / f"{name}.bin"),
                                         {torch.bfloat16: np.int16, torch.float32: np.float32}
                                         .get(dtype, np.uint8)))
        return v if dtype == torch.float32 else v.view(dtype).reshape(rows, cols)

    got = {"h": out("h", torch.bfloat16), "y": out("y", torch.bfloat16), "rstd": out("rstd", torch.float32)}
    check_norm(x, r, 0.25, n, 7, got, gamma, "from C")
    h = got["h"]
    q = {"y": out("q", torch.float8_e4m3fn), "scale": out("scale", torch.float32)}
    check_norm(h, None, 0.0, n, 0, q, gamma, "from C", "row")
    back = {"dx": out("dx", torch.bfloat16), "dresidual": out("dres", torch.bfloat16),
            "dgamma": out("dgamma", torch.float32)}
    check_backward(h, gamma, dy, 0.25, n, 7, back, dy, got["rstd"], "from C")
    want = ref.dropout(back["dresidual"], 0.25, n, 7)
    ref.assert_near(out("drop", torch.bfloat16), want,
                    ref.dropout_bound(back["dresidual"], 0.25, None, want, torch.bfloat16), "dropout in place")
    assert EPS == 1e-5  # the program's
