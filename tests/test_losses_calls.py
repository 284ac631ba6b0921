"""The drafter's losses: refusals, planners, and the definitions the GPU tests compare with."""
import itertools

import numpy as np
import pytest

from tests.losses_reference import distill_truth


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_14_gb300 import build
    build.build()
    import speculative_decoding_verification_14_gb300 as pkg
    return pkg


def test_distill_worked_examples():
    z = np.log([.5, .3, .15, .05])
    # a list that holds everything, equal to the draft: nothing to lose
    t = distill_truth(z, z, [0, 1, 2, 3], tail=True)
    assert abs(t["loss"]) < 1e-12 and np.abs(t["grad"]).max() < 1e-12
    # one token: cross entropy
    t = distill_truth(z, [0.0], [2])
    assert abs(t["loss"] + np.log(.15)) < 1e-12
    np.testing.assert_allclose(t["grad"], [.5, .3, -.85, .05], atol=1e-12)
    # two tokens renormalised, 3 : 1
    t = distill_truth(z, np.log([.6, .2]) - 5.0, [0, 1])
    assert abs(t["loss"] - (.75 * np.log(.75 / .5) + .25 * np.log(.25 / .3))) < 1e-12
    np.testing.assert_allclose(t["grad"], [-.25, .05, .15, .05], atol=1e-12)
    # the tail: .2 of the teacher against .2 of the draft, .6 and .2 against .5 and .3
    t = distill_truth(z, np.log([.6, .2]), [0, 1], tail=True)
    assert abs(t["loss"] - (.6 * np.log(.6 / .5) + .2 * np.log(.2 / .3))) < 1e-12
    np.testing.assert_allclose(t["grad"], [-.1, .1, 0, 0], atol=1e-12)
    assert distill_truth(z, [0.0, 0.0], [1, 1])["status"] == 4
    assert distill_truth(z, [0.0], [4])["status"] == 4
    assert distill_truth(z, [np.nan], [1])["status"] == 5
    assert distill_truth(z, [np.nan], [-1])["loss"] == 0.0


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T", [.5, 1.0, 3.0])
def test_distill_gradient_is_the_losses_slope(tail, T):
    rng = np.random.default_rng(5)
    z = 2 * rng.standard_normal(40)
    x = rng.permutation(40)[:7]
    a = np.log(rng.dirichlet(np.ones(9))[:7])
    g = distill_truth(z, a, x, T, tail)["grad"]
    h = 1e-5
    for v in range(40):
        e = np.zeros(40)
        e[v] = h
        slope = (distill_truth(z + e, a, x, T, tail)["loss"] - distill_truth(z - e, a, x, T, tail)["loss"]) / (2 * h)
        assert abs(slope - g[v]) < 1e-8


@pytest.mark.parametrize("B,rows,V,dtype", list(itertools.product(
    [1, 3, 64, 256, 5000], [1, 5, 33], [1, 7, 4099, 32000, 128256, 151936, 884733], [0, 1])))
def test_distill_plans(sv, B, rows, V, dtype):
    rc, p = sv.spec_distill_plan_for(152, 16, B, rows, V, dtype)
    assert rc == sv.SV_OK
    C, s, E = p["cluster"], p["slice"], 8 if dtype else 4
    assert 1 <= C <= 16 and p["grid"] == B * rows * C
    assert s % E == 0 and s * C >= V + E - 1 and p["smem_bytes"] == s // E * 16 <= 216 * 1024
    for c in (1, 3, 16):
        rc, p = sv.spec_distill_plan_for(152, 16, B, rows, V, dtype, c)
        # a slice that a CTA cannot hold
        assert rc == (sv.SV_ERR_UNSUPPORTED if -(-(-(-(V + E - 1) // E)) // c) * 16 > 216 * 1024 else sv.SV_OK)
        assert rc or p["cluster"] == c


def test_distill_plans_refuse(sv):
    for bad in ((0, 16, 1, 1, 10, 0), (152, 0, 1, 1, 10, 0), (152, 16, 0, 1, 10, 0), (152, 16, 1, 0, 10, 0),
                (152, 16, 1, 34, 10, 0), (152, 16, 1, 1, 0, 0), (152, 16, 1, 1, 1 << 31, 0), (152, 16, 1, 1, 10, 2),
                (152, 16, 1, 1, 10, 0, 17), (152, 16, 1, 1, 10, 0, -1)):
        assert sv.spec_distill_plan_for(*bad)[0] == sv.SV_ERR_INVALID_ARG, bad
    assert sv.spec_distill_plan_for(152, 8, 1, 1, 10, 0, 16)[0] == sv.SV_ERR_UNSUPPORTED
    assert sv.spec_distill_plan_for(152, 16, 1, 1, 884734, 0)[0] == sv.SV_ERR_UNSUPPORTED
    assert sv.spec_distill_plan_for(152, 16, 1, 1, 1769465, 1)[0] == sv.SV_OK
    assert sv.spec_distill_plan_for(152, 16, 1, 1, 1769466, 1)[0] == sv.SV_ERR_UNSUPPORTED


def test_null_context_is_refused(sv):
    assert sv.spec_distill_run(None, 16, 0, 10, 16, 16, 1, None, 1, 1, 10, 1.0, 0, None, 16) == sv.SV_ERR_INVALID_ARG
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_distill_get_plan(None, 1, 1, 10, 0)


@pytest.mark.gpu
def test_distill_refusals_launch_nothing(sv):
    """Every argument that is checked, one at a time out of a call that would be taken."""
    import torch
    B, rows, V, n = 2, 3, 64, 4
    lg = torch.zeros(B, rows, V, device="cuda")
    out = torch.full((B, rows, V), -7.0, device="cuda")
    fl = torch.full((B, rows, n), -7.0, device="cuda")
    tok = torch.full((B, rows, n), -7, device="cuda", dtype=torch.int32)
    ints = torch.full((B * rows,), -7, device="cuda", dtype=torch.int32)
    with sv.Verifier(4, 4, 100) as v:
        good = dict(ctx=v.ctx, logits_ptr=lg.data_ptr(), dtype=0, logits_stride=V, top_logprobs_ptr=fl.data_ptr(),
                    top_tokens_ptr=tok.data_ptr(), n=n, accept_len_ptr=None, B=B, rows_per_seq=rows, V=V, T=1.0, tail=0,
                    grad_loss_ptr=fl.data_ptr(), loss_ptr=fl.data_ptr(), grad_logits_ptr=out.data_ptr(), grad_stride=V,
                    status_ptr=ints.data_ptr())
        for bad in (dict(logits_ptr=None), dict(logits_ptr=lg.data_ptr() + 2), dict(dtype=2), dict(logits_stride=V - 1),
                    dict(logits_stride=1 << 41), dict(B=0), dict(B=5), dict(rows_per_seq=0), dict(rows_per_seq=6),
                    dict(V=0), dict(V=101), dict(status_ptr=ints.data_ptr() + 1), dict(top_logprobs_ptr=None),
                    dict(top_tokens_ptr=None), dict(top_tokens_ptr=tok.data_ptr() + 2), dict(n=0), dict(n=129),
                    dict(top_logprobs_ptr=fl.data_ptr() + 1), dict(accept_len_ptr=ints.data_ptr() + 1), dict(T=0.0),
                    dict(T=float("nan")), dict(T=float("inf")), dict(T=-1.0), dict(T=1e-31), dict(T=2e30), dict(tail=2),
                    dict(grad_loss_ptr=fl.data_ptr() + 1), dict(loss_ptr=fl.data_ptr() + 2),
                    dict(loss_ptr=None, grad_logits_ptr=None), dict(grad_logits_ptr=out.data_ptr() + 2),
                    dict(grad_stride=V - 1), dict(grad_stride=1 << 41), dict(grad_logits_ptr=lg.data_ptr(), grad_stride=V + 1),
                    dict(grad_logits_ptr=lg.data_ptr() + 4), dict(grad_logits_ptr=lg.data_ptr() + 4 * V)):
            assert sv.spec_distill_run(**{**good, **bad}) == sv.SV_ERR_INVALID_ARG, bad
        torch.cuda.synchronize()
        assert all((t == -7).all() for t in (out, fl, tok, ints)) and (lg == 0).all()
        assert v.error() == (0, 0)


@pytest.mark.gpu
def test_the_wrapper_refuses_what_the_library_cannot_see(sv):
    import torch
    with sv.Verifier(4, 4, 100) as v:
        lg = torch.zeros(2, 3, 64, device="cuda")
        a, x = torch.zeros(2, 3, 5, device="cuda"), torch.zeros(2, 3, 5, device="cuda", dtype=torch.int32)
        for bad in (lambda: v.distill(lg.cpu(), a, x), lambda: v.distill(lg, a.cpu(), x), lambda: v.distill(lg, a, x.cpu()),
                    lambda: v.distill(lg, a, x.long()), lambda: v.distill(lg, a.double(), x), lambda: v.distill(lg, a[..., :4], x),
                    lambda: v.distill(lg, a, x[..., 0]), lambda: v.distill(lg[..., ::2], a, x),
                    lambda: v.distill(lg.transpose(0, 1), a, x), lambda: v.distill(lg, a[..., ::2], x[..., ::2]),
                    lambda: v.distill(lg, a, x, torch.ones(3, device="cuda", dtype=torch.int32)),
                    lambda: v.distill(lg, a, x, grad_loss=torch.ones(2, device="cuda")),
                    lambda: v.distill(lg, a, x, out={"loss": torch.zeros(2, device="cuda")}),
                    lambda: v.distill(lg, a, x, out={"grad_logits": lg.bfloat16()})):
            with pytest.raises((ValueError, TypeError)):
                bad()
        with pytest.raises(TypeError):
            v.distill(lg.half(), a, x)
        for bad in (dict(temperature=0.0), dict(loss=False, grad=False)):
            with pytest.raises(sv.SpecVerifyError):
                v.distill(lg, a, x, **bad)


def test_cross_entropy_worked_example():
    import torch
    from tests.losses_reference import cross_entropy_truth
    # logits (0, ln 3): p = (1/4, 3/4)
    h = torch.tensor([[1.0, 2.0]], dtype=torch.float64)
    W = torch.tensor([[0.0, 0.0], [np.log(3.0), 0.0]], dtype=torch.float64)
    t = cross_entropy_truth(h, W, torch.tensor([0]), torch.tensor([2.0]))
    assert abs(t["loss"].item() - np.log(4.0)) < 1e-12 and abs(t["lse"].item() - np.log(4.0)) < 1e-12
    np.testing.assert_allclose(t["grad_hidden"].numpy(), [[2 * .75 * np.log(3.0), 0.0]], atol=1e-12)
    np.testing.assert_allclose(t["grad_weight"].numpy(), [[-1.5, -3.0], [1.5, 3.0]], atol=1e-12)


def test_cross_entropy_reference_is_autograds():
    import torch
    from tests.losses_reference import cross_entropy_truth
    g = torch.Generator().manual_seed(3)
    h, W = (torch.randn(n, 6, dtype=torch.float64, generator=g, requires_grad=True) for n in (5, 9))
    y, w = torch.randint(0, 9, (5,), generator=g), torch.rand(5, dtype=torch.float64, generator=g)
    loss = torch.nn.functional.cross_entropy(h @ W.T, y, reduction="none")
    (loss * w).sum().backward()
    t = cross_entropy_truth(h.detach(), W.detach(), y, w)
    torch.testing.assert_close(t["loss"], loss.detach())
    torch.testing.assert_close(t["grad_hidden"], h.grad)
    torch.testing.assert_close(t["grad_weight"], W.grad)


@pytest.mark.parametrize("B,rows,V,D", list(itertools.product([1, 64, 1024, 30000], [1, 8, 33],
                                                              [1, 257, 32000, 151936], [1, 64, 1000, 4096])))
def test_cross_entropy_workspaces(sv, B, rows, V, D):
    """Room for what a call keeps: packed rows, and a piece's probabilities and the gradient's sums, or a tile's
    statistics; and never that of whole logits."""
    R, pad = B * rows, -(-B * rows // 256) * 256
    rc, loss = sv.spec_cross_entropy_workspace_for(152, B, rows, V, D, 0)
    assert rc == sv.SV_OK
    packed = 2 * pad * -(-D // 8) * 8
    tiles = -(-V // 256)
    assert packed + 8 * pad * tiles <= loss < packed + 8 * pad * tiles + 16 * pad + 4096
    rc, both = sv.spec_cross_entropy_workspace_for(152, B, rows, V, D, 1)
    assert rc == sv.SV_OK and both >= loss
    piece = max(1 << 28, pad * 512)
    sums = 4 * pad * -(-D // 8) * 8
    assert both <= max(loss, packed + min(piece, 512 * pad * tiles) + 32 * sums + 32 * pad + 4096)
    if R >= 76 * 256:  # enough tiles without splits
        assert both <= max(loss, packed + piece + sums + 32 * pad + 4096)


def test_cross_entropy_workspaces_refuse(sv):
    for bad in ((0, 1, 1, 10, 8, 0), (152, 0, 1, 10, 8, 0), (152, 1, 0, 10, 8, 0), (152, 1, 34, 10, 8, 0), (152, 1, 1, 0, 8, 0),
                (152, 1, 1, 1 << 31, 8, 0), (152, 1, 1, 10, 0, 0), (152, 1, 1, 10, (1 << 20) + 1, 0), (152, 1, 1, 10, 8, 2),
                (152, 1 << 20, 2, 10, 8, 0)):
        assert sv.spec_cross_entropy_workspace_for(*bad)[0] == sv.SV_ERR_INVALID_ARG, bad
    assert sv.spec_cross_entropy_run(None, 16, 1, 8, 16, 8, 16, None, 1, 1, 10, 8, 16, 16, None, 256, 1 << 30) == \
        sv.SV_ERR_INVALID_ARG
    assert sv.spec_cross_entropy_grad(None, 16, 1, 8, 16, 8, 16, None, 16, None, 1, 1, 10, 8, 16, 8, 16, 8, None, 256,
                                      1 << 30) == sv.SV_ERR_INVALID_ARG
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_cross_entropy_workspace(None, 1, 1, 10, 8, 0)


@pytest.mark.gpu
def test_cross_entropy_refusals_launch_nothing(sv):
    import torch
    B, rows, V, D = 2, 3, 64, 16
    h = torch.zeros(B, rows, D, device="cuda", dtype=torch.bfloat16)
    W = torch.zeros(V, D, device="cuda", dtype=torch.bfloat16)
    y = torch.zeros(B, rows, device="cuda", dtype=torch.int32)
    fl = torch.full((2, B, rows), -7.0, device="cuda")
    ints = torch.full((B, rows), -7, device="cuda", dtype=torch.int32)
    gh, gw = torch.full_like(h, -7.0), torch.full_like(W, -7.0)
    with sv.Verifier(4, 4, 100) as v:
        ws = v.cross_entropy_workspace(B, rows, V, D)
        ws.fill_(0x5a)
        head = dict(ctx=v.ctx, hidden_ptr=h.data_ptr(), dtype=1, hidden_stride=D, weight_ptr=W.data_ptr(), weight_stride=D,
                    labels_ptr=y.data_ptr(), accept_len_ptr=None, B=B, rows_per_seq=rows, V=V, D=D,
                    status_ptr=ints.data_ptr(), workspace_ptr=ws.data_ptr(), workspace_bytes=ws.numel())
        shared = [dict(hidden_ptr=None), dict(hidden_ptr=h.data_ptr() + 1), dict(dtype=2), dict(hidden_stride=D - 1),
                  dict(hidden_stride=1 << 41), dict(weight_ptr=None), dict(weight_ptr=W.data_ptr() + 2),
                  dict(weight_stride=D - 8), dict(weight_stride=D + 1), dict(weight_stride=(1 << 32) + 8),
                  dict(labels_ptr=None), dict(labels_ptr=y.data_ptr() + 1), dict(accept_len_ptr=y.data_ptr() + 2),
                  dict(B=0), dict(B=5), dict(rows_per_seq=0), dict(rows_per_seq=6), dict(V=0), dict(V=101), dict(D=0),
                  dict(D=(1 << 20) + 1), dict(status_ptr=ints.data_ptr() + 1), dict(workspace_ptr=None),
                  dict(workspace_ptr=ws.data_ptr() + 16), dict(workspace_bytes=100)]
        run = dict(head, loss_ptr=fl[0].data_ptr(), lse_ptr=fl[1].data_ptr())
        for bad in shared + [dict(loss_ptr=None), dict(lse_ptr=None), dict(loss_ptr=fl.data_ptr() + 2),
                             dict(lse_ptr=fl.data_ptr() + 1)]:
            assert sv.spec_cross_entropy_run(**{**run, **bad}) == sv.SV_ERR_INVALID_ARG, bad
        assert sv.spec_cross_entropy_run(**{**run, "dtype": 0}) == sv.SV_ERR_UNSUPPORTED
        grad = dict(head, lse_ptr=fl[0].data_ptr(), grad_loss_ptr=fl[1].data_ptr(), grad_hidden_ptr=gh.data_ptr(),
                    grad_hidden_stride=D, grad_weight_ptr=gw.data_ptr(), grad_weight_stride=D)
        for bad in shared + [dict(lse_ptr=None), dict(lse_ptr=fl.data_ptr() + 2), dict(grad_loss_ptr=fl.data_ptr() + 1),
                             dict(grad_hidden_ptr=None, grad_weight_ptr=None), dict(grad_hidden_ptr=gh.data_ptr() + 1),
                             dict(grad_weight_ptr=gw.data_ptr() + 1), dict(grad_hidden_stride=D - 1),
                             dict(grad_weight_stride=D - 1), dict(grad_weight_stride=1 << 41),
                             dict(grad_hidden_ptr=h.data_ptr()), dict(grad_hidden_ptr=h.data_ptr() + 2),
                             dict(grad_weight_ptr=W.data_ptr()), dict(grad_weight_ptr=W.data_ptr() + 2 * D * (V - 1))]:
            assert sv.spec_cross_entropy_grad(**{**grad, **bad}) == sv.SV_ERR_INVALID_ARG, bad
        assert sv.spec_cross_entropy_grad(**{**grad, "dtype": 0}) == sv.SV_ERR_UNSUPPORTED
        torch.cuda.synchronize()
        assert all((t == -7).all() for t in (fl, ints, gh, gw)) and (ws == 0x5a).all()
        assert v.error() == (0, 0)
        for bad in (lambda: v.cross_entropy(h.cpu(), W, y), lambda: v.cross_entropy(h, W.cpu(), y),
                    lambda: v.cross_entropy(h, W, y.long()), lambda: v.cross_entropy(h, W[:, :8], y),
                    lambda: v.cross_entropy(h, W.T, y), lambda: v.cross_entropy(h, W, y[:1]),
                    lambda: v.cross_entropy(h.transpose(0, 1), W, y), lambda: v.cross_entropy(h.float(), W, y),
                    lambda: v.cross_entropy(h, W.float(), y), lambda: v.cross_entropy(h[..., ::2], W[:, :8], y),
                    lambda: v.cross_entropy(h, W, y, workspace=ws.cpu()), lambda: v.cross_entropy(h, W, y, workspace=fl),
                    lambda: v.cross_entropy(h, W, y, y[0, :2].clone().long()),
                    lambda: v.cross_entropy_grad(h, W, y, fl[0].double()),
                    lambda: v.cross_entropy_grad(h, W, y, fl[0], out={"grad_hidden": gh.float()}),
                    lambda: v.cross_entropy_grad(h, W, y, fl[0], out={"grad_weight": gw[:9]})):
            with pytest.raises((ValueError, TypeError)):
                bad()
        for bad in (dict(hidden_grad=False, weight_grad=False), dict(workspace=ws[:64])):
            with pytest.raises(sv.SpecVerifyError):
                v.cross_entropy_grad(h, W, y, fl[0], **bad)
