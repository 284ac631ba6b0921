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


@pytest.mark.parametrize("V", [2, 300, 4001, 32000])
@pytest.mark.parametrize("shift", [0.0, 40.0, -40.0])
def test_the_labels_gradient_keeps_its_digits(V, shift):
    """Given the losses, every d_v to its rounding to bfloat16 (2^-8 of itself) and what float32 leaves: p_v of an lse
    below 64 2^-18, its power 2^-22 and 3 |z - lse| 2^-24 with |z - lse| below 40; the label's REL and expm1's 2^-22.
    All below 2^-15."""
    import torch
    h, W, y, z, loss, lse = sure(V, shift, V + 1)
    v = gh.verifier()
    out = v.cross_entropy(h, W, y)
    w = 0.5 + torch.rand(len(y), device="cuda", generator=torch.Generator(device="cuda").manual_seed(V))
    got = v.cross_entropy_grad(h, W, y, out["lse"], grad_loss=w, loss=out["loss"], status=True)
    d = torch.exp(z - lse[:, None])
    d.scatter_(1, y.long()[:, None], torch.expm1(-loss)[:, None])
    want = (w.double()[:, None] * d).T
    err = ((got["grad_weight"][:, :len(y)].double() - want) / want).abs()
    assert err.max() <= 2.0 ** -8 + 2.0 ** -15, err.max().item()
    assert (got["grad_weight"][:, len(y):] == 0).all() and (got["status"] == 0).all()


def test_losses_given_to_ordinary_rows():
    """The gradients' own bounds hold with the losses as without; rows of a NaN loss are errors of their own."""
    import torch
    import speculative_decoding_verification_14_gb300 as sv
    from tests.test_gpu_cross_entropy import check, make
    for B, rows, V, D in ((1, 1, 1, 8), (4, 8, 1000, 128), (37, 3, 5003, 1000), (17, 16, 2000, 136)):
        h, W, y, w = make(B, rows, V, D, V + 5)
        with sv.Verifier(64, 32, 6000) as v:
            out = v.cross_entropy(h, W, y)
            check(out, v.cross_entropy_grad(h, W, y, out["lse"], grad_loss=w, loss=out["loss"]), h, W, y, w)
            lens = torch.full((B,), rows - 1, device="cuda", dtype=torch.int32)
            loss = out["loss"].clone()
            loss[0, 0] = float("nan")
            if rows > 1:
                live = torch.arange(rows, device="cuda")[None].expand(B, rows) < rows - 1
                live = live.clone()
                live[0, 0] = False
                got = v.cross_entropy_grad(h, W, y, out["lse"], lens, grad_loss=w, loss=loss, status=True)
                assert got["status"][0, 0] == 5 and torch.isnan(got["grad_hidden"][0, 0]).all() and v.error()[0] == 5
                got["grad_hidden"][0, 0] = 0
                check(None, got, h, W, y, w, live)


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


def test_refusals_of_losses():
    import torch
    import speculative_decoding_verification_14_gb300 as sv
    h, W, y, z, loss, lse = sure(300, 0.0, 3, rows=8)
    v = gh.verifier()
    f = lse.float()
    for bad in (loss, loss.float()[:4], loss.float().cpu(), torch.zeros(16, device="cuda")[::2]):
        with pytest.raises(ValueError):
            v.cross_entropy_grad(h, W, y, f, loss=bad)
    ws = v.cross_entropy_workspace(8, 1, 300, 64)
    out = torch.full_like(W, 7.0)
    assert sv.spec_cross_entropy_grad_of_loss(v.ctx, h.data_ptr(), 1, 64, W.data_ptr(), 64, y.data_ptr(), None, f.data_ptr(),
                                              f.data_ptr() + 2, None, 8, 1, 300, 64, None, 0, out.data_ptr(), 64, None,
                                              ws.data_ptr(), ws.numel()) == sv.SV_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert (out == 7.0).all()
