"""The head's cross entropy against its definition in 64 bits (tests/losses_reference.py, which derives the
tolerances); outputs are then rounded once to their types."""
import threading

import numpy as np
import pytest

from tests import gpu_helpers as gh
from tests.losses_reference import HALF, cross_entropy_truth

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def make(B, rows, V, D, seed, lean=3.0):
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = (2.0 / D ** 0.5 * torch.randn(V, (D + 7) // 8 * 8, device="cuda", generator=g)).bfloat16()[:, :D]
    y = torch.randint(0, V, (B, rows), device="cuda", generator=g, dtype=torch.int32)
    h = torch.randn(B, rows, D, device="cuda", generator=g)
    h = (h + lean * torch.rand(B, rows, 1, device="cuda", generator=g) * W[y.long()].float()).bfloat16()
    w = 0.1 + torch.rand(B, rows, device="cuda", generator=g)
    return h, W, y, w


def near(got, want, tol, half, where):
    torch = _torch()
    err = (got.double() - want).abs()
    tol = tol + half * (want.abs() + tol) + 2.0 ** -125
    bad = ~(err <= tol)
    assert not bad.any(), f"{where}: {int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[0].tolist()}: " \
                          f"{got[bad][0].item()} for {want[bad][0].item()}, allowed {tol[bad][0].item()}"


def check(out, grads, h, W, y, w=None, live=None, where=""):
    torch = _torch()
    B, rows, D = h.shape
    live = torch.ones(B, rows, dtype=torch.bool, device="cuda") if live is None else live
    at = live.view(-1).nonzero()[:, 0]
    where = f"{where} {B}x{rows} V={W.shape[0]} D={D}"
    flat = lambda t: t.reshape(B * rows, *t.shape[2:])
    t = cross_entropy_truth(flat(h)[at].double(), W.double(), flat(y)[at].long(), None if w is None else flat(w)[at])
    if out is not None:
        assert (out["status"] == 0).all(), where
        for k in ("loss", "lse"):
            near(flat(out[k])[at], t[k], t[k + "_tol"], HALF["f32"], f"{where} {k}")
            assert (out[k][~live] == 0).all(), where
    if grads is not None and "grad_hidden" in grads:
        near(flat(grads["grad_hidden"])[at], t["grad_hidden"], t["grad_hidden_tol"], HALF["bf16"], f"{where} grad_hidden")
        assert (grads["grad_hidden"][~live] == 0).all(), where
    if grads is not None and "grad_weight" in grads:
        near(grads["grad_weight"], t["grad_weight"], t["grad_weight_tol"], HALF["bf16"], f"{where} grad_weight")


def both(v, h, W, y, lens=None, w=None, **kw):
    out = v.cross_entropy(h, W, y, lens, **kw)
    return out, v.cross_entropy_grad(h, W, y, out["lse"], lens, grad_loss=w, **kw)


SIZES = [(1, 1, 256, 64), (1, 1, 1, 8), (2, 1, 7, 16), (3, 3, 300, 72), (4, 8, 1000, 128), (16, 16, 512, 64),
         (16, 16, 513, 200), (17, 16, 2000, 136), (37, 3, 5003, 1000), (8, 5, 32000, 1024), (100, 8, 4096, 512),
         (64, 4, 20011, 333)]


@pytest.mark.parametrize("B,rows,V,D", SIZES)
def test_loss(B, rows, V, D):
    h, W, y, w = make(B, rows, V, D, V + D)
    v = gh.verifier()
    check(v.cross_entropy(h, W, y), None, h, W, y)
    assert v.error() == (0, 0)


@pytest.mark.parametrize("B,rows,V,D", SIZES)
def test_gradients(B, rows, V, D):
    h, W, y, w = make(B, rows, V, D, V + D + 1)
    v = gh.verifier()
    out, grads = both(v, h, W, y, w=w)
    check(out, grads, h, W, y, w)
    assert v.error() == (0, 0)
