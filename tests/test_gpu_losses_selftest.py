"""What the losses' kernels do behind a wait that ran out: spec_losses_selftest has them take one of their waits, once
it is over, for one that did.  No wait really runs out, so every call below has to be quick: a drain that
missed a copy would take its ten seconds."""
import time

import pytest

from tests.test_gpu_cross_entropy import both, check, make

pytestmark = pytest.mark.gpu

TIMEOUT = 6
# pairs with several tiles to come and fills in flight; few rows of few tiles; pieces of the vocabulary; rows on no 16 bytes
SIZES = [(40, 8, 60000, 1024), (2, 3, 700, 72), (130, 32, 40000, 72), (5, 30, 900, 333)]


def timed(f):
    import torch
    torch.cuda.synchronize()
    t = time.perf_counter()
    out = f()
    torch.cuda.synchronize()
    assert time.perf_counter() - t < 1.0
    return out


def case(B, rows, V, D):
    import torch
    h, W, y, w = make(B, rows, V, D, V + 7)
    y[0, 0], y[-1, -1] = -1, V  # a row that does not count and one in error
    live = torch.ones(B, rows, dtype=torch.bool, device="cuda")
    live[0, 0] = live[-1, -1] = False
    return h, W, y, w, live


@pytest.mark.parametrize("B,rows,V,D", SIZES)
def test_losses(B, rows, V, D):
    import torch
    import speculative_decoding_verification_14_gb300 as sv
    h, W, y, w, live = case(B, rows, V, D)
    with sv.Verifier(256, 32, 60000) as v:
        ws = v.cross_entropy_workspace(B, rows, V, D)
        timed(lambda: v.cross_entropy(h, W, y, workspace=ws))
        good = timed(lambda: v.cross_entropy(h, W, y, workspace=ws))
        assert v.error()[1] == 1 << 4
        assert sv.spec_losses_selftest(v.ctx, sv.SV_SELFTEST_LOGITS) == 0
        out = timed(lambda: v.cross_entropy(h, W, y, workspace=ws))
        assert v.error()[1] == (1 << 4 | 1 << TIMEOUT)
        assert torch.isnan(out["loss"][live]).all() and torch.isnan(out["lse"][live]).all()
        assert (out["status"][live] == TIMEOUT).all()
        assert out["loss"][0, 0] == 0 and out["status"][0, 0] == 0 and out["status"][-1, -1] == 4
        assert sv.spec_losses_selftest(v.ctx, sv.SV_SELFTEST_OFF) == 0
        again = timed(lambda: v.cross_entropy(h, W, y, workspace=ws))
        assert all(torch.equal(again[k].nan_to_num(), good[k].nan_to_num()) for k in good) and v.error()[1] == 1 << 4


@pytest.mark.parametrize("B,rows,V,D", SIZES)
@pytest.mark.parametrize("product", ["PROBS", "HIDDEN", "WEIGHT"])
def test_gradients(product, B, rows, V, D):
    import torch
    import speculative_decoding_verification_14_gb300 as sv
    h, W, y, w, live = case(B, rows, V, D)
    with sv.Verifier(256, 32, 60000) as v:
        ws = v.cross_entropy_workspace(B, rows, V, D)
        out = v.cross_entropy(h, W, y, workspace=ws)
        call = lambda **kw: timed(lambda: v.cross_entropy_grad(h, W, y, out["lse"], grad_loss=w, workspace=ws, status=True, **kw))
        call()
        good = call()
        v.error()
        assert sv.spec_losses_selftest(v.ctx, getattr(sv, "SV_SELFTEST_" + product)) == 0
        for kw in ({}, {"hidden_grad": False}, {"weight_grad": False}):
            if product == "HIDDEN" and "hidden_grad" in kw or product == "WEIGHT" and "weight_grad" in kw:
                continue  # that product is not among the call's
            got = call(**kw)
            assert v.error()[1] == (1 << 4 | 1 << TIMEOUT)
            assert (got["status"][live] == TIMEOUT).all() and got["status"][0, 0] == 0 and got["status"][-1, -1] == 4
            if "grad_hidden" in got:
                assert torch.isnan(got["grad_hidden"][live]).all() and (got["grad_hidden"][0, 0] == 0).all()
            if "grad_weight" in got:
                lost = torch.isnan(got["grad_weight"])
                assert lost[:min(V, 256), :min(D, 256)].all()
                if product == "PROBS" or product == "HIDDEN" and V < 40000:  # one piece: its last product is left out as a whole
                    assert lost.all()
        assert sv.spec_losses_selftest(v.ctx, sv.SV_SELFTEST_OFF) == 0
        again = call()
        assert all(torch.equal(again[k].nan_to_num(), good[k].nan_to_num()) for k in good) and v.error()[1] == 1 << 4
        check(None, {k: t.nan_to_num() for k, t in again.items()}, h, W, y, w, live)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cluster,V", [(0, 2000), (3, 4003), (16, 5001)])
@pytest.mark.parametrize("wait", ["COPY", "EXCHANGE"])
def test_distillation(wait, cluster, V, dtype):
    """The middle row's cluster loses that row and those it takes after it; every other row is as it was."""
    import torch
    import speculative_decoding_verification_14_gb300 as sv
    from tests.test_gpu_distill import make as rows_of
    B, rows = 1024, 4
    z, a, x, w = rows_of(B, rows, V, 12, dtype, V)
    lens = torch.randint(0, rows + 1, (B,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(V),
                         dtype=torch.int32)
    lens[B // 2] = rows
    live = (torch.arange(rows, device="cuda")[None] < lens[:, None]).view(-1)
    mid = B * rows // 2
    with sv.Verifier(B, rows, V) as v:
        v.set_plan_override(cluster)
        call = lambda: timed(lambda: v.distill(z, a, x, lens, tail=True, grad_loss=w))
        call()
        good = call()
        assert v.error() == (0, 0)
        assert sv.spec_losses_selftest(v.ctx, getattr(sv, "SV_SELFTEST_DISTILL_" + wait)) == 0
        out = call()
        assert v.error()[1] == 1 << TIMEOUT
        assert sv.spec_losses_selftest(v.ctx, sv.SV_SELFTEST_OFF) == 0
        again = call()
        assert all(torch.equal(again[k], good[k]) for k in good) and v.error() == (0, 0)
    loss, st, g = out["loss"].view(-1), out["status"].view(-1), out["grad_logits"].view(B * rows, V)
    bad = st == TIMEOUT
    lost = bad.nonzero()[:, 0].tolist()
    # of the row itself an exchange's wait is lost in the last CTA alone
    nan = torch.isnan(g).any(-1)
    assert nan[mid] and (wait == "EXCHANGE" or lost[0] == mid) and lost[0] >= mid and len(lost) > 1
    step = min(b - a for a, b in zip(lost, lost[1:]))
    assert all((r - mid) % step == 0 for r in lost) and live[lost].all()
    assert live[mid::step].sum() == len(lost) + (lost[0] != mid)
    assert torch.isnan(loss[bad]).all() and torch.isnan(g[bad]).all()
    rest = ~bad
    rest[mid] = False
    assert torch.equal(loss[rest], good["loss"].view(-1)[rest]) and (st[rest] == 0).all()
    assert torch.equal(g[rest], good["grad_logits"].view(B * rows, V)[rest])


def test_refusals():
    import speculative_decoding_verification_14_gb300 as sv
    assert sv.spec_losses_selftest(None, 0) == sv.SV_ERR_INVALID_ARG
    with sv.Verifier(4, 4, 100) as v:
        for bad in (-1, 100):
            assert sv.spec_losses_selftest(v.ctx, bad) == sv.SV_ERR_INVALID_ARG
