"""Distillation from top log-probabilities against its definition in 64 bits (tests/losses_reference.py, which
derives the tolerances); the results are then rounded once to the outputs' types."""
import threading

import numpy as np
import pytest

from tests import gpu_helpers as gh
from tests.losses_reference import HALF, distill_truth

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def make(B, rows, V, n, dtype, seed, spread=2.5, T=1.0):
    """Draft rows, and a teacher near them, as top lists of it."""
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = (spread * torch.randn(B, rows, V, device="cuda", generator=g)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    t = (z.float() + 0.8 * torch.randn(z.shape, device="cuda", generator=g)) / T
    n0 = min(n, V)
    top = t.log_softmax(-1).topk(n0, dim=-1)
    a, x = torch.full((B, rows, n), float("nan"), device="cuda"), torch.full((B, rows, n), -1, device="cuda", dtype=torch.int32)
    a[..., :n0], x[..., :n0] = top.values, top.indices.to(torch.int32)
    w = 0.1 + torch.rand(B, rows, device="cuda", generator=g)
    return z, a, x, w


def check(out, z, a, x, T=1.0, tail=False, w=None, lens=None, dtype="f32"):
    B, rows, _ = z.shape
    z, a, x = z.double().cpu().numpy(), a.double().cpu().numpy(), x.cpu().numpy()
    w = np.ones((B, rows)) if w is None else w.cpu().numpy()
    loss, st = out["loss"].cpu().numpy(), out["status"].cpu().numpy()
    grad = out["grad_logits"].double().cpu().numpy() if "grad_logits" in out else None
    for b in range(B):
        for i in range(rows):
            where = f"row {b},{i} of V={z.shape[-1]} n={x.shape[-1]} T={T} tail={tail}"
            if lens is not None and i >= int(lens[b]):
                assert loss[b, i] == 0 and st[b, i] == 0 and (grad is None or (grad[b, i] == 0).all()), where
                continue
            t = distill_truth(z[b, i], a[b, i], x[b, i], T, tail, w[b, i])
            assert st[b, i] == t["status"], where
            if t["status"]:
                assert np.isnan(loss[b, i]) and (grad is None or np.isnan(grad[b, i]).all()), where
                continue
            np.testing.assert_allclose(loss[b, i], t["loss"], rtol=HALF["f32"], atol=t["loss_tol"], err_msg=where)
            if grad is not None:
                err = np.abs(grad[b, i] - t["grad"])
                tol = t["grad_tol"] + HALF[dtype] * (np.abs(t["grad"]) + t["grad_tol"]) + 2.0 ** -125
                bad = np.flatnonzero(~(err <= tol))
                assert not len(bad), f"{where}: entry {bad[0]} of {len(bad)}: {grad[b, i][bad[0]]} for " \
                                     f"{t['grad'][bad[0]]}, allowed {tol[bad[0]]}"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("B,rows,V,n,T", [(1, 1, 1, 1, 1.0), (2, 2, 2, 1, 1.0), (3, 1, 7, 3, 0.5), (2, 3, 8, 8, 1.0),
                                          (2, 3, 9, 20, 2.0), (4, 2, 33, 5, 1.0), (5, 3, 1000, 20, 0.7), (3, 2, 4099, 128, 1.0),
                                          (37, 3, 5003, 33, 0.8), (2, 5, 32000, 20, 1.0), (1, 2, 50257, 100, 1.3),
                                          (1, 1, 128256, 20, 1.0), (1, 2, 151936, 64, 0.6)])
def test_rows(B, rows, V, n, T, tail, dtype):
    z, a, x, w = make(B, rows, V, n, dtype, 7 * V + n, T=T)
    out = gh.verifier().distill(z, a, x, temperature=T, tail=tail, grad_loss=w)
    check(out, z, a, x, T, tail, w, dtype=dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cluster", [1, 2, 3, 5, 8, 16])
def test_every_plan(cluster, dtype):
    """Clusters with empty, partial and full last slices."""
    v = gh.verifier()
    v.set_plan_override(cluster)
    try:
        for V in (1, 15, 100, 20011):
            z, a, x, w = make(3, 2, V, 24, dtype, V, T=0.9)
            for tail in (False, True):
                check(v.distill(z, a, x, temperature=0.9, tail=tail, grad_loss=w), z, a, x, 0.9, tail, w, dtype=dtype)
    finally:
        v.set_plan_override(0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_longest_rows(dtype):
    torch = _torch()
    V = 884733 if dtype == "f32" else 1769465
    z, a, x, w = make(1, 1, V, 30, dtype, 3)
    z[0, 0, V - 1] = 20.0  # listed or not, the last entry counts
    check(gh.verifier().distill(z, a, x, tail=True, grad_loss=w), z, a, x, 1.0, True, w, dtype=dtype)


def test_rows_of_lengths_and_lists():
    """Rows from accept_len on are not read; a row without an entry has no loss, whatever it holds."""
    torch = _torch()
    z, a, x, w = make(6, 4, 3001, 12, "f32", 11)
    lens = torch.tensor([1, 4, 2, 3, 0, 4], device="cuda", dtype=torch.int32)
    dead = torch.arange(4, device="cuda")[None] >= lens[:, None]
    z[dead], a[dead], x[dead], w[dead] = float("nan"), float("nan"), 1 << 30, float("nan")
    x[1, 2], z[1, 2] = -1, float("nan")
    x[3, 0, 1:], a[3, 0, 1:] = -1, float("inf")
    x[5, 1, ::2], a[5, 1, ::2] = -1, float("nan")
    for tail in (False, True):
        out = gh.verifier().distill(z, a, x, lens, tail=tail, grad_loss=w)
        check(out, z, a, x, 1.0, tail, w, lens.cpu())
        assert out["loss"][1, 2] == 0 and (out["grad_logits"][1, 2] == 0).all()
    assert gh.verifier().error() == (0, 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_logits(dtype):
    """-inf and the type's lowest value, off the list and on it; a tail that vanishes beside one entry."""
    torch = _torch()
    V, n = 2050, 8
    z, a, x, w = make(8, 1, V, n, dtype, 13)
    low = torch.finfo(z.dtype).min
    off = torch.ones(8, V, device="cuda", dtype=torch.bool).scatter_(1, x[:, 0].long(), False)
    z[0, 0] = torch.where(off[0], -torch.inf, z[0, 0])  # no mass off the list
    z[1, 0] = torch.where(off[1], low, z[1, 0])
    a[:2] = (a[:2] - a[:2].logsumexp(-1, keepdim=True))  # the list holds all the mass, but for rounding
    z[2, 0, ::3] = -torch.inf
    z[3, 0, 1::3] = low
    z[4, 0, x[4, 0, 0].long()] = -torch.inf  # the teacher's best is masked: infinitely wrong
    z[5, 0, x[5, 0, 0].long()] = low
    z[6, 0, x[6, 0, 0].long()] = 200.0  # the tail's weights are below any float beside it
    a[6, 0, 1:] = -torch.inf
    a[6, 0, 0] = -0.5
    z[7] = low
    z[7, 0, 5] = -torch.inf
    for tail in (False, True):
        out = gh.verifier().distill(z, a, x, tail=tail, grad_loss=w)
        check(out, z, a, x, 1.0, tail, w, dtype=dtype)
        assert torch.isinf(out["loss"][4]).all() and torch.isfinite(out["grad_logits"]).all()


def test_errors_stay_in_their_rows():
    torch = _torch()
    import speculative_decoding_verification_14_gb300 as sv
    for dtype in ("f32", "bf16"):
        z, a, x, w = make(14, 1, 3000, 9, dtype, 17)
        z[1, 0, 2999] = float("nan")
        z[2, 0, 0] = float("inf")
        z[3] = -torch.inf
        x[4, 0, 3] = 3000
        x[5, 0, 8] = -2
        x[6, 0, 2] = x[6, 0, 7]
        a[7, 0, 0] = float("nan")
        a[8, 0, 4] = float("inf")
        a[9] = -torch.inf  # no teacher at all; under tail all of it is the rest
        z[10, 0, x[10, 0, 1].long()] = float("nan")
        x[11] = 1 << 30
        z[12, 0, x[12, 0, 0].long()] = float("inf")
        with sv.Verifier(20, 1, 4000) as v:
            for tail in (False, True):
                out = v.distill(z, a, x, tail=tail, grad_loss=w)
                check(out, z, a, x, 1.0, tail, w, dtype=dtype)
                assert out["status"][:, 0].tolist() == [0, 5, 5, 5, 4, 4, 4, 5, 5, 0 if tail else 5, 5, 4, 5, 0]
                assert v.error() == (4, 1 << 4 | 1 << 5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_alignment_and_in_place(dtype):
    torch = _torch()
    v = gh.verifier()
    B, rows, V, n = 3, 2, 1003, 10
    z, a, x, w = make(B, rows, V, n, dtype, 19)
    want = v.distill(z, a, x, tail=True, grad_loss=w)
    check(want, z, a, x, 1.0, True, w, dtype=dtype)

    def laid(stride, start):
        flat = torch.full((B * rows * stride + 16,), 77.0, device="cuda", dtype=z.dtype)
        return flat, flat[start:start + B * rows * stride].view(B, rows, stride)[..., :V]
    for stride in (1003, 1004, 1007, 1024):
        for start in (0, 1, 3):
            zf, zv = laid(stride, start)
            zv.copy_(z)
            for gs, g0 in ((stride, start), (stride, 2), (1016, 0)):
                gf, gv = laid(gs, g0)
                out = {"loss": torch.empty_like(want["loss"]), "grad_logits": gv, "status": torch.empty_like(want["status"])}
                v.distill(zv, a, x, tail=True, grad_loss=w, out=out)
                check(out, z, a, x, 1.0, True, w, dtype=dtype)
                gv.fill_(77.0)
                assert (gf == 77.0).all()  # nothing beside the rows is written
            out = {"loss": torch.empty_like(want["loss"]), "grad_logits": zv, "status": torch.empty_like(want["status"])}
            v.distill(zv, a, x, tail=True, grad_loss=w, out=out)
            check(out, z, a, x, 1.0, True, w, dtype=dtype)
            zv.fill_(77.0)
            assert (zf == 77.0).all()


def test_parts_of_a_call_and_repeats_agree():
    torch = _torch()
    v = gh.verifier()
    z, a, x, w = make(9, 3, 32001, 20, "bf16", 23)
    both = v.distill(z, a, x, tail=True, grad_loss=w)
    again = v.distill(z, a, x, tail=True, grad_loss=w)
    loss = v.distill(z, a, x, tail=True, grad=False)
    grad = v.distill(z, a, x, tail=True, grad_loss=w, loss=False, status=False)
    assert set(loss) == {"loss", "status"} and set(grad) == {"grad_logits"}
    for k in both:
        assert torch.equal(both[k], again[k])
    assert torch.equal(both["loss"], loss["loss"]) and torch.equal(both["grad_logits"], grad["grad_logits"])
    ones = v.distill(z, a, x, tail=True)
    assert torch.equal(ones["grad_logits"], v.distill(z, a, x, tail=True, grad_loss=torch.ones_like(w))["grad_logits"])
    # rows of their own, and two dimensions
    flat = v.distill(z.view(27, -1), a.view(27, -1), x.view(27, -1), tail=True, grad_loss=w.view(27))
    assert torch.equal(flat["loss"].view(9, 3), both["loss"])
    torch.testing.assert_close(flat["grad_logits"].view(z.shape).float(), both["grad_logits"].float(), rtol=2 ** -7, atol=1e-9)


@pytest.mark.parametrize("tail", [False, True])
def test_the_gradient_is_the_losses_slope(tail):
    """Against differences of the call's own losses: a step h of every logit.  Either loss is off by the
    reference's bound and a rounding, its third derivative is below 1."""
    torch = _torch()
    v = gh.verifier()
    V, n, h = 50, 6, 2.0 ** -6
    z, a, x, _ = make(1, 1, V, n, "f32", 29, spread=1.0)
    z = (z * 256).round() / 256  # steps of h are exact
    grad = v.distill(z, a, x, tail=tail)["grad_logits"][0, 0]
    step = torch.eye(V, device="cuda")[:, None] * h
    up, down = (v.distill(z.expand(V, 1, V) + d, a.expand(V, 1, n).contiguous(), x.expand(V, 1, n).contiguous(),
                          tail=tail, grad=False)["loss"][:, 0] for d in (step, -step))
    t = distill_truth(z[0, 0].double().cpu().numpy(), a[0, 0].double().cpu().numpy(), x[0, 0].cpu().numpy(), 1.0, tail)
    off = 2 * t["loss_tol"] + 2.0 ** -24 * (t["loss"] + h)
    assert ((up.double() - down.double()) / (2 * h) - grad.double()).abs().max() < off / h + h * h / 6


def test_a_teacher_from_a_verify():
    """Target rows -> log-probabilities of the emitted rows -> the drafter's loss and gradient, on a stream, then
    captured and replayed on other data."""
    torch = _torch()
    v = gh.verifier()
    B, K1, V, n, T = 10, 4, 8009, 20, 0.8
    g = torch.Generator(device="cuda").manual_seed(31)

    def rows():
        t = 2.5 * torch.randn(B, K1, V, device="cuda", generator=g)
        return t.bfloat16(), (t + torch.randn(t.shape, device="cuda", generator=g)).bfloat16()
    target, z = rows()
    u = torch.rand(B, K1, device="cuda", generator=g)
    tokens = v.sample(z[:, :K1 - 1].contiguous(), u[:, :K1 - 1].contiguous(), temperature=T)["tokens"]
    w = torch.rand(B, K1, device="cuda", generator=g)

    def step():
        ver = v.run_draft_logits(target, z[:, :K1 - 1].contiguous(), tokens, u, T, T)
        lp = v.logprobs(target, ver["out_tokens"], ver["accept_len"], temperature=T, top_n=n)
        return ver, lp, v.distill(z, lp["top_logprobs"], lp["top_tokens"], ver["accept_len"], temperature=T, tail=True,
                                  grad_loss=w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ver, lp, out = step()
    s.synchronize()
    assert 1 < int(ver["accept_len"].min()) + int(ver["accept_len"].max()) and int(ver["accept_len"].sum()) < B * K1
    check(out, z, lp["top_logprobs"], lp["top_tokens"], T, True, w, ver["accept_len"].cpu(), "bf16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ver, lp, out = step()
    for _ in range(2):
        t2, z2 = rows()
        target.copy_(t2)
        z.copy_(z2)
        graph.replay()
        torch.cuda.synchronize()
        check(out, z, lp["top_logprobs"], lp["top_tokens"], T, True, w, ver["accept_len"].cpu(), "bf16")


def test_two_threads_on_streams_of_their_own():
    torch = _torch()
    import speculative_decoding_verification_14_gb300 as sv
    jobs = [make(4, 3, 16001, 20, "f32", s) for s in (41, 42)]
    want = [gh.verifier().distill(z, a, x, tail=True, grad_loss=w) for z, a, x, w in jobs]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            z, a, x, w = jobs[i]
            with sv.Verifier(8, 4, 20000) as v, torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    out = v.distill(z, a, x, tail=True, grad_loss=w)
                    torch.cuda.current_stream().synchronize()
                    assert all(torch.equal(out[k], want[i][k]) for k in out)
        except BaseException as e:  # handed to the test's own thread
            failed.append(e)
    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cluster,V", [(0, 3001), (4, 9011), (3, 4003)])
def test_more_rows_than_run_at_once(cluster, V, dtype):
    """Clusters take row after row: live ones, ones behind the last, ones without a list and erroneous ones."""
    torch = _torch()
    v = gh.verifier()
    B, rows = 260, 4
    z, a, x, w = make(B, rows, V, 12, dtype, V)
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = torch.randint(0, rows + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
    lens[100:180] = 0  # many in turn that a CTA has nothing to do for
    x[::7, 0] = -1
    z[::11, 1, V - 1] = float("nan")
    x[::13, 2, 3] = x[::13, 2, 9]
    v.set_plan_override(cluster)
    try:
        for tail in (False, True):
            out = v.distill(z, a, x, lens, tail=tail, grad_loss=w)
            check(out, z, a, x, 1.0, tail, w, lens.cpu(), dtype)
    finally:
        v.set_plan_override(0)
        v.error()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_entries_far_above_the_rest(dtype):
    """Off the list, where no thread's first vector lies, and so far that a sum against those overflows."""
    torch = _torch()
    V = 40000
    z, a, x, w = make(6, 1, V, 16, dtype, 53, spread=1.0)
    for i, (at, top) in enumerate([(39999, 12.0), (39999, 40.0), (30011, 200.0), (17777, 3e4), (39990, 3e38)]):
        z[i, 0, at] = top
    z[5, 0, :20000] = -float("inf")  # a slice without a logit in its first vectors
    for tail in (False, True):
        check(gh.verifier().distill(z, a, x, tail=tail, grad_loss=w), z, a, x, 1.0, tail, w, dtype=dtype)


@pytest.mark.parametrize("T", [2.0 ** -100, 1e-3, 0.05, 50.0, 1e6, 2.0 ** 100])
def test_temperatures(T):
    for dtype in ("f32", "bf16"):
        z, a, x, w = make(4, 2, 5001, 16, dtype, 61, T=max(T, 0.3))
        for tail in (False, True):
            out = gh.verifier().distill(z, a, x, temperature=T, tail=tail, grad_loss=w)
            check(out, z, a, x, T, tail, w, dtype=dtype)


def test_offsets_beyond_32_bits():
    """17000 rows of 128256: their last rows, in place."""
    torch = _torch()
    v = gh.verifier()
    B, V = 17000, 128256
    z, a, x, w = make(2, 1, V, 20, "bf16", 59)
    big = torch.zeros(B, 1, V, device="cuda", dtype=torch.bfloat16)
    big[-2:] = z
    ab, xb = a[:1].expand(B, 1, 20).contiguous(), x[:1].expand(B, 1, 20).contiguous()
    ab[-2:], xb[-2:] = a, x
    wb = torch.ones(B, 1, device="cuda")
    wb[-2:] = w
    out = {"loss": torch.empty(B, 1, device="cuda"), "grad_logits": big,
           "status": torch.empty(B, 1, device="cuda", dtype=torch.int32)}
    v.distill(big, ab, xb, tail=True, grad_loss=wb, out=out)
    check({k: t[-2:] for k, t in out.items()}, z, a, x, 1.0, True, w, dtype="bf16")
    check({k: t[:1] for k, t in out.items()}, torch.zeros_like(z[:1]), a[:1], x[:1], 1.0, True, None, dtype="bf16")
    assert (out["status"] == 0).all() and torch.equal(out["loss"][:-2], out["loss"][:1].expand(B - 2, 1))
