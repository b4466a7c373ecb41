"""A CTA of a cluster whose peer gave up: in a test-only build of the staged gradients the
first CTA of each cluster stops at its first row, before it has sent the row's statistics.
The other CTAs have sent theirs and wait for the merge until their own budget (about a
second) is over; then the cluster ends, the call's timeout is recorded and the context is
usable."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FR_DEVERR_TIMEOUT = 2


def child(lib_path: str) -> None:
    sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]
    import torch
    import logits_ref as ref
    import reduction_pointwise_row_gb300 as fr
    fr.library_path = lambda: lib_path
    rows = 16  # clusters of 8 of them are on the device at once
    x = (3 * torch.randn(rows, 130001, generator=torch.Generator().manual_seed(1))).bfloat16()
    t = torch.arange(rows)
    g = torch.ones(1)
    i, z = t[:, None].cuda(), torch.zeros(rows, 1, device="cuda")
    res = {}
    v, tc, gc = x.cuda(), t.cuda(), g.cuda()
    fr.fr_xent_backward(v, tc, gc, form="split")
    res["xent"] = fr.fr_check_device_error()
    fr.fr_distill_backward(v, i, z, gc, form="split")
    res["distill"] = fr.fr_check_device_error()
    got = fr.fr_xent_backward(v, tc, gc, form="looped")
    r = ref.xent_backward(x, t, g)
    ref.assert_near(got["dlogits"], r, ref.gradient_bound(x, r, g), "after the timeouts")
    res["after"] = fr.fr_check_device_error()
    print(json.dumps(res), flush=True)


def test_a_cluster_whose_first_cta_gives_up_ends():
    from reduction_pointwise_row_gb300 import buildlib
    lib = buildlib.build_variant("peer_wait_test", ["-DFR_TEST_GRAD_WAIT_RUNS_OUT=2"],
                                 recompile=("logit_grad.cu",))
    r = subprocess.run([sys.executable, os.path.abspath(__file__), lib], capture_output=True,
                       text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stdout + r.stderr
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert res == {"xent": FR_DEVERR_TIMEOUT, "distill": FR_DEVERR_TIMEOUT, "after": 0}, res


if __name__ == "__main__":
    child(sys.argv[1])
