"""How near the losses and gradients come, as a whole, to 64 bits: norms of the error, and losses near 0, where bounds that
add every rounding's size (tests/losses_reference.py) see nothing.

Distillation's sums, for those bounds: 224 threads walk a slice of at most 13824 vectors, 62 each, a vector's weights in 4
additions, and join as integers, so that 66 roundings of 2^-24 and the integers' last places (2^-38 a thread) are less than the
128 of 2^-24 allowed there.

Distillation's loss in two floats: powers 2^-28, logarithms 2^-29 (tests/test_losses_arithmetic.py), products and sums below 2^-44.
Of loss = sum t (a - ln q) + r (ln r - ln q_rest) the shares' errors meet again in r = 1 - sum t: 2^-28; the listed weights' are
2^-28 of S; three logarithms 3 x 2^-29: 3.5 x 2^-28 in all, 2^-26 allowed.  The weights off the list are float32 powers, 2^-22
of themselves: what they move S by and what they move q_rest by cancels but for |q_rest - r|, which is below the loss's own
size (Pinsker: (q_rest - r)^2 <= loss / 2, and here 2^-22 sqrt(loss / 2) is below 2^-27); without a tail their mass
is itself below the loss.  Rounding the loss: 2^-24 of it.

The head's gradients: d is rounded to bfloat16, 2^-8 of itself at worst, which a gradient of one large d inherits whole; the
output's rounding is uniform in half a unit, 1.7e-3 in the mean square over a binade: sqrt(2^-16 + 1.7e-3^2) = 4.3e-3 and
1e-4 for float32 sums.  The losses: a tensor core adds 16 products at a time and may cut, each step up to 2^-23 of
the partial sum: over D / 16 steps of a partial sum that grows to the logit, a mean of half of that, D 2^-28 of a logit's size
at worst, with lse and z_y cut alike; 2e-7 for powers, sums and logarithms."""
import numpy as np
import pytest

from tests import gpu_helpers as gh
from tests.losses_reference import distill_truth

pytestmark = pytest.mark.gpu


def teacher(z, n, T, noise, g):
    """Lists of a target that is the draft but for `noise`."""
    import torch
    t = z.double() / T + noise * torch.randn(z.shape, device="cuda", generator=g, dtype=torch.float64)
    top = t.log_softmax(-1).topk(n, dim=-1)
    return top.values.float(), top.indices.to(torch.int32)


def truths(z, a, x, T, tail):
    z, a, x = z.double().cpu().numpy(), a.double().cpu().numpy(), x.cpu().numpy()
    return [distill_truth(z[i, 0], a[i, 0], x[i, 0], T, tail) for i in range(len(z))]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V,n,T", [(1000, 20, 0.7), (32000, 20, 1.0), (50257, 64, 0.8), (151936, 100, 1.3)])
def test_distillation_as_a_whole(V, n, T, tail, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(V)
    z = (2.5 * torch.randn(24, 1, V, device="cuda", generator=g)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    a, x = teacher(z, n, T, 0.8, g)
    out = gh.verifier().distill(z, a, x, temperature=T, tail=tail)
    want = truths(z, a, x, T, tail)
    loss = np.array([t["loss"] for t in want])
    got = out["loss"][:, 0].double().cpu().numpy()
    assert np.linalg.norm(got - loss) <= 5e-7 * np.linalg.norm(loss)
    grad = np.stack([t["grad"] for t in want])
    err = out["grad_logits"][:, 0].double().cpu().numpy() - grad
    # bfloat16: uniform in half a unit, 1.7e-3 over a binade, at worst sqrt(1/3) of 2^-8 for a gradient just above a power of two
    assert np.linalg.norm(err) <= (5e-7 if dtype == "f32" else 2.3e-3) * np.linalg.norm(grad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("noise", [2e-3, 5e-3, 1.2e-2])
@pytest.mark.parametrize("V,n,T", [(1000, 20, 1.0), (32000, 64, 0.8), (128256, 128, 1.0)])
def test_distillations_small_losses(V, n, T, noise, dtype):
    """A drafter that has nearly learned its target: with a tail, and without one where the list holds all but nothing."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(n)
    z = 2.5 * torch.randn(24, 1, V, device="cuda", generator=g)
    peaked = torch.randn(24, 1, V, device="cuda", generator=g)
    peaked[:, :, ::V // n] += 30.0
    for tail, rows in ((True, z), (False, peaked)):
        rows = rows.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
        a, x = teacher(rows, n, T, noise, g)
        loss = np.array([t["loss"] for t in truths(rows, a, x, T, tail)])
        assert 1e-8 < loss.max() < 3e-4 and loss.min() > 0
        got = gh.verifier().distill(rows, a, x, temperature=T, tail=tail, grad=False)["loss"][:, 0].double().cpu().numpy()
        assert (np.abs(got - loss) <= 2.0 ** -26 + 2.0 ** -21 * loss).all(), np.abs(got - loss).max()


@pytest.mark.parametrize("B,rows,V,D", [(40, 5, 32000, 1024), (128, 8, 20011, 4096), (130, 32, 40000, 512), (8, 5, 32000, 1024)])
def test_a_head_as_a_whole(B, rows, V, D):
    """One size per kind of call: a row tile, several, several pieces of the vocabulary, few rows."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(D)
    R = B * rows
    W = (2.0 / D ** 0.5 * torch.randn(V, D, device="cuda", generator=g)).bfloat16()
    y = torch.randint(0, V, (B, rows), device="cuda", generator=g, dtype=torch.int32)
    h = torch.randn(B, rows, D, device="cuda", generator=g)
    h = (h + 4.0 * torch.rand(B, rows, 1, device="cuda", generator=g) * W[y.long()].float()).bfloat16()
    w = (0.5 + 0.5 * torch.rand(B, rows, device="cuda", generator=g)) / R
    v = gh.verifier()
    out = v.cross_entropy(h, W, y)
    grads = {given: v.cross_entropy_grad(h, W, y, out["lse"], grad_loss=w, loss=out["loss"] if given else None)
             for given in (False, True)}
    hd, Wd, yd = h.view(R, D).double(), W.double(), y.view(R, 1).long()
    lse, loss = torch.empty(R, 1, device="cuda", dtype=torch.float64), torch.empty(R, 1, device="cuda", dtype=torch.float64)
    gh64, gw64 = torch.empty_like(hd), torch.zeros_like(Wd)
    for at in torch.arange(R, device="cuda").split(512):
        z = hd[at] @ Wd.T
        lse[at] = torch.logsumexp(z, -1, keepdim=True)
        loss[at] = lse[at] - z.gather(1, yd[at])
        d = torch.exp(z - lse[at])
        d.scatter_(1, yd[at], torch.expm1(-loss[at]))
        d *= w.view(R, 1)[at].double()
        gh64[at] = d @ Wd
        gw64 += d.T @ hd[at]
    norm = lambda got, want: ((got.reshape(want.shape).double() - want).norm() / want.norm()).item()
    bound = 2e-7 + D * 2.0 ** -28
    assert norm(out["loss"], loss) <= bound and norm(out["lse"], lse) <= bound
    for got in grads.values():
        assert norm(got["grad_hidden"], gh64) <= 4.4e-3 and norm(got["grad_weight"], gw64) <= 4.4e-3
    print(B, rows, V, D, norm(out["loss"], loss), norm(out["lse"], lse), norm(got["grad_hidden"], gh64), norm(got["grad_weight"], gw64))
