"""Rows that a head already gets right: losses of 1e-6 to 1e-4, where a sum that begins with the label's weight keeps
no digit of the rest.

Hidden state r is the r-th unit vector, so that the logits are the weight's own bfloat16 values, exact in any order
of summing, and the head's gradient at [v, r] is row r's d_v.

What float32 may be off by, relative to s = sum of the others' weights against the label's: a weight's power 2^-22
and 3 ln 2 |y| 2^-24 for y binades below the running maximum; a sum is multiplied by such powers again at each of a
tile's eight steps where the maximum grows and once where tiles join; Y binades from the lowest to the largest
that counts come to 3 ln 2 (2 Y) 2^-24 for all of them, and ten powers to 10 x 2^-22; 8 + 2 additions of a step, 8 of
a tile, 1 of the join (two floats); exp(m - z_y) 2^-22 and |m - z_y| 2^-24; log1p 2^-23, two products and the
rounding of the result: with Y <= 24 and |m - z_y| <= 20, (40 + 100 + 19 + 4 + 20 + 2 + 3) 2^-24 = 188 x 2^-24."""
import pytest

from tests import gpu_helpers as gh

pytestmark = pytest.mark.gpu

REL = 188 * 2.0 ** -24


def sure(V, shift, seed, rows=48):
    """Rows whose label holds all but 1e-6 to 1e-4 of the mass, logits about `shift`."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    D = 64
    z = (shift + 1.5 * torch.randn(rows, V, device="cuda", generator=g)).clamp(shift - 7, shift + 7).bfloat16().double()
    y = torch.randint(0, V, (rows,), device="cuda", generator=g)
    z.scatter_(1, y[:, None], float("-inf"))
    rest = torch.logsumexp(z, -1)
    want = 10.0 ** -(4 + 2 * torch.rand(rows, device="cuda", generator=g, dtype=torch.float64))
    z.scatter_(1, y[:, None], (rest - want.log())[:, None].bfloat16().double())
    W = torch.zeros(V, D, device="cuda", dtype=torch.bfloat16)
    W[:, :rows] = z.T.bfloat16()
    h = torch.eye(D, device="cuda", dtype=torch.bfloat16)[:rows]
    loss = torch.log1p(torch.exp(rest - z.gather(1, y[:, None])[:, 0]))
    return h.contiguous(), W, y.int(), z, loss, torch.logsumexp(z, -1)


@pytest.mark.parametrize("V", [2, 300, 4001, 32000])
@pytest.mark.parametrize("shift", [0.0, 40.0, -40.0])
def test_losses_keep_their_digits(V, shift):
    h, W, y, z, loss, lse = sure(V, shift, V)
    assert loss.max() < 2e-4 and loss.min() > 1e-7
    out = gh.verifier().cross_entropy(h, W, y)
    err = ((out["loss"].double() - loss) / loss).abs()
    assert err.max() <= REL, err.max().item()
    assert ((out["lse"].double() - lse).abs() <= 2.0 ** -24 * lse.abs() + REL * loss).all()
    assert (out["status"] == 0).all()


def test_labels_and_others_that_are_nothing():
    """A label's logit of -inf: infinitely wrong; all the others' -inf: nothing to lose; the label's NaN or +inf: an
    error; a head of one token."""
    import torch
    import speculative_decoding_verification_14_gb300 as sv
    inf = float("inf")
    h, W, y, z, loss, lse = sure(600, 0.0, 5, rows=5)
    for r, v in ((0, -inf), (2, float("nan")), (3, inf)):
        W[int(y[r]), r] = v
    W[:, 1] = -inf
    W[int(y[1]), 1] = 3.0
    W[:, 4] = -inf
    # products with a hidden state's zeros would be NaN: a row at a time, the others' columns left out
    with sv.Verifier(8, 1, 1000) as v:
        got = [v.cross_entropy(h[r:r + 1, r:r + 1].repeat(1, 8), torch.nn.functional.pad(W[:, r:r + 1], (0, 7)), y[r:r + 1])
               for r in range(5)]
        assert v.error()[1] == 1 << sv.SV_ERR_NONFINITE
    L, S, E = ([o[k].item() for o in got] for k in ("loss", "status", "lse"))
    assert S == [0, 0, 5, 5, 5] and L[0] == inf and abs(E[0] - torch.logsumexp(z[0].scatter(0, y[:1].long(), -inf), 0).item()) < 1e-5
    assert L[1] == 0.0 and E[1] == 3.0 and all(x != x for x in (*L[2:], *E[2:]))
    one = gh.verifier().cross_entropy(h, W[:1, :].nan_to_num(0, 0, 0).contiguous(), torch.zeros_like(y))
    assert (one["loss"] == 0).all() and (one["status"] == 0).all()
