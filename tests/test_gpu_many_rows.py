"""The head's cross entropy over more rows than a batch has: which rows count, and where they are packed."""
import pytest

from tests import gpu_helpers as gh

pytestmark = pytest.mark.gpu


def rows_of(B, rows, V, D, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = torch.randn(V, D, device="cuda", generator=g).bfloat16()
    h = torch.randn(B, rows, D, device="cuda", generator=g).bfloat16()
    y = torch.randint(-1, V, (B, rows), device="cuda", generator=g, dtype=torch.int32)
    return h, W, y


@pytest.mark.parametrize("lengths", [False, True])
@pytest.mark.parametrize("B,rows", [(64, 32), (2049, 1), (100, 30), (1024, 8), (2731, 3), (513, 16), (20000, 7)])
def test_which_rows_count(B, rows, lengths):
    """Either side of the number from which rows are counted ahead; long stretches of rows that do not count, and of ones that
    do, across what is counted together.  Each row's answer is that of a call of its own few rows."""
    import torch
    V, D = 40, 16
    v = gh.verifier()
    h, W, y = rows_of(B, rows, V, D, B)
    y.view(-1)[500:2600] = -1
    y.view(-1)[B * rows // 2: B * rows // 2 + 1300] = 3
    y.view(-1)[-1] = V - 1
    lens = torch.randint(0, rows + 1, (B,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(B),
                         dtype=torch.int32) if lengths else None
    live = y >= 0
    if lengths:
        lens[-1] = rows
        live &= torch.arange(rows, device="cuda")[None] < lens[:, None]
    out = v.cross_entropy(h, W, y, lens)
    w = torch.rand(B, rows, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    grads = v.cross_entropy_grad(h, W, y, out["lse"], lens, grad_loss=w)
    z = h.double() @ W.double().T
    lse = torch.logsumexp(z, -1)
    loss = lse - z.gather(-1, y.clamp(min=0).long()[..., None])[..., 0]
    # a logit is a float32 sum of 16 exact products (17 x 2^-23 of the sum of their sizes), lse adds 2^-20 and its rounding
    size = (h.double().abs() @ W.double().abs().T).amax(-1)
    tol = 2 * 17 * 2.0 ** -23 * size + 2.0 ** -20 + 2.0 ** -23 * (lse.abs() + z.abs().amax(-1))
    for k, want in (("loss", loss), ("lse", lse)):
        assert ((out[k].double() - want).abs() <= tol)[live].all() and (out[k][~live] == 0).all(), k
    assert (out["status"] == 0).all()
    d = torch.exp(z - lse[..., None])
    d.scatter_add_(-1, y.clamp(min=0).long()[..., None], torch.full_like(d[..., :1], -1.0))
    d = torch.where(live[..., None], d * w.double()[..., None], 0.0)
    # d off by its rounding to bfloat16 and two logits' errors; sums of V or R of them in float32, rounded to bfloat16
    off = d.abs() * 2.0 ** -8 + (d.abs() + w[..., None]) * (2 * tol)[..., None]
    gh_tol = off @ W.double().abs() * 1.01
    want = d @ W.double()
    assert ((grads["grad_hidden"].double() - want).abs() <= gh_tol + 2.0 ** -8 * (want.abs() + gh_tol))[live].all()
    assert (grads["grad_hidden"][~live] == 0).all()
    flat = lambda t: t.reshape(B * rows, -1)
    gw_tol = flat(off).T @ flat(h).double().abs() * 1.01 + 2.0 ** -12 * (flat(d).abs().T @ flat(h).double().abs())
    want = flat(d).T @ flat(h).double()
    assert ((grads["grad_weight"].double() - want).abs() <= gw_tol + 2.0 ** -8 * (want.abs() + gw_tol)).all()


def test_the_call_grows_with_its_rows():
    """2^20 rows against 2^18, with lengths: four times the rows may take eight times as long, not sixteen."""
    import torch
    v = gh.verifier()
    took = []
    for B in (1 << 14, 1 << 16):
        h, W, y = rows_of(B, 16, 64, 16, 5)
        lens = torch.full((B,), 12, device="cuda", dtype=torch.int32)
        ws = v.cross_entropy_workspace(B, 16, 64, 16, grad=False)
        out = v.cross_entropy(h, W, y, lens, workspace=ws)
        best = float("inf")
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            v.cross_entropy(h, W, y, lens, workspace=ws, out=out)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        took.append(best)
    assert took[1] < 8 * took[0], took
