"""The entry points for rows of logits from a plain C program
(tests/c_abi/logits_from_c.c, built with gcc against include/fr.h): no Python or
PyTorch in that process.  Its outputs must meet the same bounds as the binding's."""
import subprocess

import numpy as np
import pytest
import torch

import logits_ref as ref
from test_c_abi_gpu import build_c_program
from test_logits_gpu import check_logprobs, loss_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def c_logits(tmp_path_factory):
    return build_c_program("logits_from_c", tmp_path_factory)


@pytest.mark.parametrize("rows,cols,top", [(300, 9000, 20), (5, 40001, 3), (2, 200, 128)])
def test_logits_from_a_c_program(c_logits, tmp_path, rows, cols, top):
    r = np.random.default_rng(11)
    x = torch.from_numpy(r.normal(0, 3, (rows, cols)).astype(np.float32)).bfloat16()
    t = torch.from_numpy(r.integers(0, cols, rows))
    t[1] = -100
    i = torch.from_numpy(r.integers(0, cols, (rows, top)))
    z = torch.from_numpy(r.normal(0, 2, (rows, top)).astype(np.float32))
    g = torch.from_numpy(r.normal(0, 1, rows).astype(np.float32))
    for name, v in (("x", x.view(torch.int16)), ("t", t), ("i", i), ("z", z), ("g", g)):
        v.numpy().tofile(str(tmp_path / f"{name}.bin"))
    p = subprocess.run([c_logits, str(rows), str(cols), str(top), str(tmp_path)],
                       capture_output=True, text=True, timeout=120)
    assert p.returncode == 0, p.stderr

    def out(name, dtype=np.float32):
        v = torch.from_numpy(np.fromfile(str(tmp_path / f"{name}.bin"), dtype))
        return v.view(torch.bfloat16).reshape(rows, cols) if dtype == np.int16 else v

    got = {"logprob": out("logprob"), "entropy": out("entropy"), "lse": out("lse"),
           "top_index": out("top", np.int64).reshape(rows, top)}
    check_logprobs(x, got, t, top, "from C")
    w = ref.xent(x, t)
    ref.assert_near(out("loss"), w, ref.eps(cols) + 4 * ref.U * w.abs(), "loss")
    w = ref.xent_backward(x, t, g)
    ref.assert_near(out("xent", np.int16), w, ref.gradient_bound(x, w, g), "xent gradient")
    w = ref.distill(x, i, z, 2.0)
    for name in ("distill", "distill_step"):
        ref.assert_near(out(name), w, loss_bound(x, w, i, z, 2.0), name)
    w = ref.distill_backward(x, i, z, g, 2.0)
    q, _, _ = ref.teacher(i, z, 2.0)
    dense = torch.zeros_like(w).scatter_add_(1, i, q)
    b = ref.gradient_bound(x, w, g * 2, temperature=2.0)
    ref.assert_near(out("distill_grad", np.int16), w,
                    b + 2 * g.double().abs()[:, None] * dense * 160 * ref.U, "its gradient")
    w = ref.logprobs_backward(x, t, g, g)
    ref.assert_near(out("logprobs_grad", np.int16), w, ref.gradient_bound(x, w, g, g),
                    "gradient in place")
