"""A wait of the staged gradient kernel that runs out records FR_DEVERR_TIMEOUT and
the kernel returns.

Every wait of that kernel is bounded (about one second for a copy that takes
microseconds), so this test uses a test-only build of the library in which a CTA's
wait for its first row runs out at once, most often while its copy is in flight.  The CTA's workers stop together, its helpers copy nothing more and wait
for the copies they issued before, and the CTA ends.  The build runs in a child
process; there the call must report the timeout, one CTA per row and a cluster
per row alike, and calls of other kernels of the same library must then be right,
which shows that the context is usable."""
import json
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FR_DEVERR_TIMEOUT = 2


def child(lib_path: str) -> None:
    sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]
    import logits_ref as ref
    import reduction_pointwise_row_gb300 as fr
    fr.library_path = lambda: lib_path
    x = (3 * torch.randn(64, 30000, generator=torch.Generator().manual_seed(1))).bfloat16()
    t = torch.arange(64)
    g = torch.ones(1)
    v, tc, gc = x.cuda(), t.cuda(), g.cuda()
    res = {}
    for form in ("persistent", "split"):
        fr.fr_xent_backward(v, tc, gc, form=form)
        res[form] = fr.fr_check_device_error()
    got = fr.fr_xent_backward(v, tc, gc, form="looped")
    r = ref.xent_backward(x, t, g)
    ref.assert_near(got["dlogits"], r, ref.gradient_bound(x, r, g), "after the timeouts")
    top = fr.fr_logprobs(v, tc, top=3)["top_index"].cpu()
    assert torch.equal(top, ref.logprobs(x, t, 3)["top_index"])
    res["after"] = fr.fr_check_device_error()
    print(json.dumps(res), flush=True)


def test_shortened_waits_time_out_and_the_kernel_returns():
    from reduction_pointwise_row_gb300 import buildlib
    lib = buildlib.build_variant("grad_wait_test", ["-DFR_TEST_GRAD_WAIT_RUNS_OUT"],
                                 recompile=("logit_grad.cu",))
    r = subprocess.run([sys.executable, os.path.abspath(__file__), lib], capture_output=True,
                       text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stdout + r.stderr
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert res == {"persistent": FR_DEVERR_TIMEOUT, "split": FR_DEVERR_TIMEOUT, "after": 0}, res


if __name__ == "__main__":
    child(sys.argv[1])
