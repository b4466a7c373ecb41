"""A residual block's row operators (fr_dropout, fr_rmsnorm, fr_rmsnorm_quant,
fr_rmsnorm_backward) without a GPU: arguments refused on the host before any CUDA
call, and the formulas that the GPU tests use against published values and
automatic differentiation."""
import ctypes
import math

import numpy as np
import pytest
import torch

import reduction_pointwise_row_gb300 as fr
import rmsnorm_ref as ref

P = ctypes.c_void_p
X, R, H, Y, G, S, N = (P(0x100000 * (i + 1)) for i in range(7))  # N: rng
ODD = P(0x100001)
BIG = 1 << 40
OK_SO_FAR = 8  # every argument accepted: without a device, FR_ERR_NO_DEVICE
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not device memory")


def dropout(x=X, residual=R, y=Y, rows=4, cols=8, ldx=8, ldr=8, ldy=8, p=0.5, rng=N, site=0, dtype=1):
    return fr.lib().fr_dropout(x, residual, y, rows, cols, ldx, ldr, ldy, p, rng, site, dtype, None)


def rmsnorm(x=X, residual=R, gamma=G, h=H, y=Y, rstd=S, rows=4, cols=8, ldx=8, ldr=8, ldh=8, ldy=8,
            eps=1e-5, p=0.5, rng=N, site=0, dtype=1, form=0):
    return fr.lib().fr_rmsnorm(x, residual, gamma, h, y, rstd, rows, cols, ldx, ldr, ldh, ldy, eps,
                               p, rng, site, dtype, form, None)


def quant(x=X, residual=R, gamma=G, h=H, y=Y, scale=S, mode=0, sr=1, sc=1, rstd=None, rows=4, cols=8,
          ldx=8, ldr=8, ldh=8, ldy=8, eps=1e-5, p=0.5, rng=N, site=0, dtype=1, form=0):
    return fr.lib().fr_rmsnorm_quant(x, residual, gamma, h, y, scale, mode, sr, sc, rstd, rows, cols,
                                     ldx, ldr, ldh, ldy, eps, p, rng, site, dtype, form, None)


def backward(dy=X, h=H, gamma=G, rstd=S, dh=R, dx=Y, dres=P(0x900000), dgamma=P(0xA00000), rows=4,
             cols=8, ld_dy=8, ld_h=8, ld_dh=8, ld_dx=8, ld_dres=8, p=0.5, rng=N, site=0, dtype=1,
             form=0, ws=P(0xB00000), nws=1 << 30):
    return fr.lib().fr_rmsnorm_backward(dy, h, gamma, rstd, dh, dx, dres, dgamma, rows, cols, ld_dy,
                                        ld_h, ld_dh, ld_dx, ld_dres, p, rng, site, dtype, form, ws,
                                        nws, None)


SHAPE = [(dict(rows=0), 1), (dict(cols=0), 1), (dict(rows=-1), 1), (dict(dtype=2), 2),
         (dict(dtype=-1), 2), (dict(p=-0.1), 1), (dict(p=1.5), 1), (dict(p=math.nan), 1),
         (dict(rng=None), 1), (dict(rng=P(0x700004)), 4)]
FORWARD = SHAPE + [
    (dict(x=None), 1), (dict(y=None), 1), (dict(ldx=7), 1), (dict(ldr=7), 1), (dict(ldy=7), 1),
    (dict(x=ODD), 4), (dict(residual=ODD), 4), (dict(x=P(0x100002), dtype=0), 4),
    (dict(rows=BIG, cols=BIG, ldx=BIG, ldr=BIG, ldy=BIG), 1),
    (dict(rows=1 << 31), 3), (dict(rows=1, cols=1 << 31, ldx=1 << 31, ldr=1 << 31, ldy=1 << 31), 3)]
NORM = [(dict(gamma=None), 1), (dict(h=None), 1), (dict(residual=None, p=0.0), 1), (dict(ldh=7), 1),
        (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1), (dict(gamma=ODD), 4),
        (dict(rstd=P(0x600002)), 4), (dict(h=ODD), 4), (dict(form=3), 3), (dict(form=-1), 3),
        (dict(cols=16392, ldx=16392, ldr=16392, ldh=16392, ldy=16392, form=1), 3),
        # overlaps: of outputs, with other strides, with vectors
        (dict(h=Y), 1), (dict(y=X, ldx=16), 1), (dict(h=P(0x100008)), 1), (dict(gamma=Y), 1),
        (dict(rstd=H), 1), (dict(rstd=P(0x500008)), 1), (dict(rng=P(0x300008)), 1)]


@pytest.mark.parametrize("call,more", [(dropout, []), (rmsnorm, NORM), (quant, NORM)])
def test_forward_arguments(call, more):
    for kw, want in FORWARD + more:
        if call is not dropout:
            kw = dict(kw)
            if kw.get("ldx", 0) >= BIG or kw.get("ldx", 0) == 1 << 31:
                kw["ldh"] = kw["ldx"]
        if call is quant and kw in (dict(y=X, ldx=16), ):
            kw = dict(y=X)  # another type: never over an input
        if call is quant and "rstd" in kw and kw["rstd"] is not H and kw["rstd"].value == 0x500008:
            kw = dict(rstd=G)  # vectors over vectors
        assert call(**kw) == want, (call.__name__, kw)


def test_dropout_overlaps():
    assert dropout(y=X, ldx=16) == 1
    assert dropout(y=P(0x100008)) == 1
    assert dropout(rng=P(0x400010)) == 1


@no_device
def test_forward_arguments_that_pass():
    assert dropout() == OK_SO_FAR
    assert dropout(p=0.0, rng=None, residual=None) == OK_SO_FAR
    assert dropout(p=1.0, y=X) == OK_SO_FAR and dropout(y=R) == OK_SO_FAR
    assert dropout(x=X, y=P(0x100010), ldx=16, ldy=16) == OK_SO_FAR  # in the gaps
    assert rmsnorm() == OK_SO_FAR and rmsnorm(rstd=None, dtype=0) == OK_SO_FAR
    assert rmsnorm(residual=None) == OK_SO_FAR and rmsnorm(p=0.0, rng=None) == OK_SO_FAR
    assert rmsnorm(residual=None, p=0.0, h=None, y=X, eps=0.0) == OK_SO_FAR
    assert rmsnorm(h=R, y=X) == OK_SO_FAR and rmsnorm(residual=X) == OK_SO_FAR
    assert quant(h=X) == OK_SO_FAR and quant(mode=2, rstd=R) == 1  # rstd over an input
    assert quant(mode=1, cols=300, ldx=300, ldr=300, ldh=300, ldy=300, sr=3) == OK_SO_FAR
    assert quant(mode=1, cols=300, ldx=300, ldr=300, ldh=300, ldy=300, sr=1, sc=4) == OK_SO_FAR
    assert quant(mode=2, sr=0, sc=0) == OK_SO_FAR
    assert backward() == OK_SO_FAR and backward(dres=None, dgamma=None, ws=None, nws=0) == OK_SO_FAR
    assert backward(p=0.0, rng=None, dres=None, dx=X) == OK_SO_FAR
    assert backward(dx=H, dres=R, dh=R) == OK_SO_FAR


def test_scale_arguments():
    wide = dict(cols=300, ldx=300, ldr=300, ldh=300, ldy=300)
    for kw in (dict(scale=None), dict(mode=3), dict(mode=-1), dict(sr=0), dict(sr=BIG << 22),
               dict(mode=1, sr=2, sc=1, **wide), dict(mode=1, sr=1, sc=3, **wide),
               dict(mode=1, sr=3, sc=3, **wide), dict(mode=1, sr=0, sc=4, **wide),
               dict(mode=1, sr=3, sc=-1, **wide), dict(scale=Y), dict(scale=H), dict(scale=G),
               dict(scale=S, rstd=S)):
        assert quant(**kw) == 1, kw
    assert quant(scale=P(0x600002)) == 4


def test_backward_arguments():
    for kw, want in SHAPE + [
            (dict(dy=None), 1), (dict(h=None), 1), (dict(gamma=None), 1), (dict(rstd=None), 1),
            (dict(dx=None), 1), (dict(ld_dy=7), 1), (dict(ld_h=7), 1), (dict(ld_dh=7), 1),
            (dict(ld_dx=7), 1), (dict(ld_dres=7), 1), (dict(dy=ODD), 4), (dict(dx=ODD), 4),
            (dict(dgamma=P(0xA00001)), 4), (dict(rstd=P(0x600001)), 4), (dict(form=3), 3),
            (dict(p=0.0, rng=None), 1),  # dresidual without dropout
            (dict(dres=Y), 1), (dict(dx=X, ld_dx=16), 1), (dict(dx=P(0x100008)), 1),
            (dict(dgamma=G), 1), (dict(dgamma=S), 1), (dict(dgamma=X), 1), (dict(dgamma=Y), 1),
            (dict(dx=G), 1), (dict(dres=S), 1), (dict(rng=P(0x400010)), 1),
            (dict(rows=1 << 31), 3)]:
        assert backward(**kw) == want, kw
    n = 16392
    long = dict(cols=n, ld_dy=n, ld_h=n, ld_dh=n, ld_dx=n, ld_dres=n)
    assert backward(form=1, rows=2, **long) == 3
    n = 8200
    long = dict(cols=n, ld_dy=n, ld_h=n, ld_dh=n, ld_dx=n, ld_dres=n)
    assert backward(form=1, rows=2, dtype=0, **long) == 3


def test_forms_and_names():
    assert fr.fr_auto_form("rmsnorm", 4, 16384, "bf16") == "persistent"
    assert fr.fr_auto_form("rmsnorm_quant", 4, 16385, "f32") == "looped"
    assert fr.fr_auto_form("rmsnorm_backward", 4, 8192, "f32") == "persistent"
    assert fr.fr_auto_form("rmsnorm_backward", 4, 8200, "f32") == "looped"
    assert fr.fr_auto_form("rmsnorm_backward", 4, 16384, "bf16") == "persistent"


def test_the_binding_refuses_host_tensors():
    x, g = torch.zeros(4, 8), torch.ones(8)
    n = torch.zeros(2, dtype=torch.int64)
    for call in (lambda: fr.fr_dropout(x, 0.5, n), lambda: fr.fr_rmsnorm(x, g),
                 lambda: fr.fr_rmsnorm_quant(x, g),
                 lambda: fr.fr_rmsnorm_backward(x, x, g, torch.ones(4))):
        with pytest.raises(ValueError):
            call()


# Known answers of Philox4x32 with 7 and 10 rounds, published with the generator.
ANSWERS = [
    (7, (0, 0, 0, 0), (0, 0), (0x5F6FB709, 0x0D893F64, 0x4F121F81, 0x4F730A48)),
    (7, (0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x5207DDC2, 0x45165E59, 0x4D8EE751, 0x8C52F662)),
    (10, (0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    (10, (0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
]


@pytest.mark.parametrize("rounds,ctr,key,want", ANSWERS)
def test_the_generator_gives_the_published_values(rounds, ctr, key, want):
    assert tuple(int(v) for v in ref.philox(ctr, key, rounds)) == want


def test_thresholds():
    assert [ref.threshold(p) for p in (0.0, 1e-9, 0.1, 0.5, 0.9999999, 1.0)] == \
        [0, 1, 6554, 32768, 65535, 65536]


def test_the_mask_drops_its_share_and_varies_with_everything():
    base = ref.keep(256, 1000, 0.3, (5, 7))[0]
    share = 1.0 - base.double().mean()
    assert abs(share - 0.3) < 5 * math.sqrt(0.21 / base.numel())
    for other in (ref.keep(256, 1000, 0.3, (6, 7))[0], ref.keep(256, 1000, 0.3, (5, 8))[0],
                  ref.keep(256, 1000, 0.3, (5, 7), 9)[0], ref.keep(257, 1000, 0.3, (5, 7))[0][1:]):
        agree = (other == base).double().mean()  # 0.7^2 + 0.3^2 of independent ones
        assert abs(agree - 0.58) < 5 * math.sqrt(0.25 / base.numel())
    assert torch.equal(ref.keep(256, 1000, 0.3, (5, 7 + 9))[0], ref.keep(256, 1000, 0.3, (5, 7), 9)[0])
    assert torch.equal(ref.keep(100, 333, 0.3, (5, 7))[0], base[:100, :333])


def test_formulas_against_automatic_differentiation():
    torch.manual_seed(2)
    x, res = (torch.randn(5, 37, dtype=torch.float64, requires_grad=True) for _ in range(2))
    gamma = torch.randn(37, dtype=torch.float64, requires_grad=True)
    dy, dh = torch.randn(5, 37, dtype=torch.float64), torch.randn(5, 37, dtype=torch.float64)
    m, f = ref.keep(5, 37, 0.4, (1, 2), 3)
    h = res + torch.where(m, x * f, 0.0)
    y, rstd = ref.norm(h, gamma, 1e-5)
    assert torch.allclose(y, torch.nn.functional.rms_norm(h, (37,), gamma, 1e-5), atol=1e-12)
    ((y * dy).sum() + (h * dh).sum()).backward()
    d, dgamma = ref.backward(dy, h.detach(), gamma.detach(), rstd.detach(), dh)
    assert torch.allclose(res.grad, d, atol=1e-12)
    assert torch.allclose(gamma.grad, dgamma, atol=1e-12)
    assert torch.allclose(x.grad, torch.where(m, d * f, 0.0), atol=1e-12)


def test_groups():
    v = torch.arange(300.0).expand(2, 300)
    s = ref.scales(v, 128)
    assert s.shape == (2, 3) and np.allclose(s[0] * 448, [127, 255, 299])


def test_a_second_thread_finds_both_lookups(monkeypatch):
    """The stream's lookup is published after the device's: a call that finds the device's
    alone resolves both."""
    monkeypatch.setattr(fr, "_current_device", lambda: 0)
    monkeypatch.setattr(fr, "_current_raw_stream", None)

    class Tensor:
        def get_device(self):
            return 0

    try:
        fr._device_of(Tensor())
    except (RuntimeError, AssertionError):
        pass  # no device here
    assert fr._current_raw_stream is not None


def elements_left(rows, row, ld, cols):
    """As the kernels bound an aligned unit's load at the end of its matrix."""
    n = (rows - 1 - row) * ld
    return 2**31 - 1 if n >= 8 else n + cols


def test_units_of_rows_in_phase_stay_within_their_matrix():
    """A whole 16-byte unit is loaded only where all of it lies between the matrix's first
    and last element, also for rows shorter than a unit."""
    for rows in (1, 2, 3, 5, 9, 20):
        for cols in (1, 2, 3, 7, 8, 9, 15, 257):
            for ld in (cols, cols + 1, cols + 5):
                total = (rows - 1) * ld + cols
                for row in range(rows):
                    phase = row * ld & 7
                    for unit in range((cols + phase + 7) // 8):
                        col = unit * 8 - phase
                        if col < cols and col <= elements_left(rows, row, ld, cols) - 8:
                            assert 0 <= row * ld + col and row * ld + col + 8 <= total


def test_algorithmic_bytes():
    from reduction_pointwise_row_gb300 import traffic
    n = 16384 * 4096
    assert traffic.algorithmic_bytes("dropout", 16384, 4096) == 4 * n
    assert traffic.algorithmic_bytes("rmsnorm", 16384, 4096, residual=True, drop=True) == \
        8 * n + 4 * (16384 + 4096)
    assert traffic.algorithmic_bytes("rmsnorm", 16384, 4096, dtype="f32") == 8 * n + 4 * (16384 + 4096)
    assert traffic.algorithmic_bytes("rmsnorm_quant", 16384, 4096, residual=True) == \
        7 * n + 4 * (16384 + 4096)
    assert traffic.algorithmic_bytes("rmsnorm_backward", 16384, 4096, residual=True, drop=True) == \
        10 * n + 4 * (2 * 4096 + 16384)
