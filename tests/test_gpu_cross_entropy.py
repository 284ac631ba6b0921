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


@pytest.mark.parametrize("B,rows,V,D", [(1, 1, 600, 64), (16, 8, 257, 72), (33, 8, 1000, 64), (8, 16, 5000, 40)])
def test_each_gradient_alone(B, rows, V, D):
    torch = _torch()
    h, W, y, w = make(B, rows, V, D, V + 3)
    v = gh.verifier()
    out, want = both(v, h, W, y, w=w)
    only = [v.cross_entropy_grad(h, W, y, out["lse"], grad_loss=w, hidden_grad=a, weight_grad=not a) for a in (True, False)]
    assert set(only[0]) == {"grad_hidden"} and set(only[1]) == {"grad_weight"}
    assert torch.equal(only[0]["grad_hidden"], want["grad_hidden"]) and torch.equal(only[1]["grad_weight"], want["grad_weight"])
    again = both(v, h, W, y, w=w)
    for k in out:
        assert torch.equal(out[k], again[0][k])
    for k in want:
        assert torch.equal(want[k], again[1][k])
    ones = torch.ones_like(w)
    a, b = (v.cross_entropy_grad(h, W, y, out["lse"], grad_loss=g) for g in (None, ones))
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_several_pieces_of_the_vocabulary():
    """A piece's probabilities stay within 256 MB: 4160 rows of 40000 are two pieces, the second one's last tile partial."""
    h, W, y, w = make(130, 32, 40000, 72, 71)
    v = gh.verifier()
    out, grads = both(v, h, W, y, w=w)
    check(out, grads, h, W, y, w)


def test_rows_that_do_not_count():
    """Behind accept_len and of label -1: whatever they hold reaches nothing; and no row at all."""
    torch = _torch()
    v = gh.verifier()
    for B, rows, V, D in ((40, 5, 3000, 136), (3, 4, 500, 64), (90, 8, 777, 72)):
        h, W, y, w = make(B, rows, V, D, 73 + B)
        g = torch.Generator(device="cuda").manual_seed(B)
        lens = torch.randint(0, rows + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
        lens[0], lens[1] = 0, rows
        y[2:, ::2] = torch.where(torch.rand(y[2:, ::2].shape, device="cuda", generator=g) < 0.3, -1, y[2:, ::2])
        dead = torch.arange(rows, device="cuda")[None] >= lens[:, None]
        live = ~dead & (y >= 0)
        h[~live], w[~live] = float("nan"), float("nan")
        y[dead] = 1 << 30
        out, grads = both(v, h, W, y, lens, w)
        check(out, grads, h, W, y, w, live)
        none = torch.full_like(y, -1)
        out, grads = both(v, h, W, none, None, w)
        assert all((t == 0).all() for t in (*out.values(), *grads.values()))
        out, grads = both(v, h, W, y, torch.zeros_like(lens), w)
        assert all((t == 0).all() for t in (*out.values(), *grads.values()))
    assert v.error() == (0, 0)


def test_errors_stay_in_their_rows():
    torch = _torch()
    import speculative_decoding_verification_14_gb300 as sv
    B, rows, V, D = 50, 2, 900, 80
    h, W, y, w = make(B, rows, V, D, 79)
    y[3, 0], y[4, 1] = V, -2
    h[5, 0, 7] = float("nan")
    h[6, 1, 79] = float("inf")
    bad = torch.zeros(B, rows, dtype=torch.bool, device="cuda")
    bad[3, 0] = bad[4, 1] = bad[5, 0] = bad[6, 1] = True
    want = torch.where(bad, 5, 0).to(torch.int32)
    want[3, 0] = want[4, 1] = 4
    with sv.Verifier(64, 4, 1000) as v:
        out, grads = both(v, h, W, y, w=w)
        assert v.error() == (4, 1 << 4 | 1 << 5)
        assert torch.equal(out["status"], want)
        assert torch.isnan(out["loss"][bad]).all() and torch.isnan(out["lse"][bad]).all()
        assert torch.isnan(grads["grad_hidden"][bad]).all()
        st = v.cross_entropy_grad(h, W, y, out["lse"], grad_loss=w, status=True)["status"]
        assert torch.equal(st, want)
        # the others' answers are those of a call without the erroneous rows
        y2 = torch.where(bad, -1, y)
        o2, g2 = both(v, h, W, y2, w=w)
        for k in ("loss", "lse"):
            assert torch.equal(out[k][~bad], o2[k][~bad])
        assert torch.equal(grads["grad_weight"], g2["grad_weight"])
        assert torch.equal(grads["grad_hidden"][~bad], g2["grad_hidden"][~bad])
        check({**o2, "status": torch.zeros_like(y)}, g2, h, W, y, w, ~bad)
        # a logit beyond float in every row
        W[17] = float("nan")
        out, grads = both(v, h, W, y2, w=w)
        assert torch.isnan(out["loss"][~bad]).all() and (out["status"][~bad] == 5).all() and (out["loss"][bad] == 0).all()
        assert (grads["grad_weight"] == 0).all() and torch.isnan(grads["grad_hidden"][~bad]).all()


def test_wide_logits():
    """Logits of some hundreds, equal ones, and a head of one token: sums against the maximum, p of 0 and 1."""
    torch = _torch()
    v = gh.verifier()
    h, W, y, w = make(9, 3, 700, 64, 83)
    big = (h * 40.0).contiguous()
    out, grads = both(v, big, W, y, w=w)
    check(out, grads, big, W, y, w)
    zero = torch.zeros_like(h)
    out, grads = both(v, zero, W, y, w=w)
    check(out, grads, zero, W, y, w)
    one = W[:1].contiguous()
    out, grads = both(v, h, one, torch.zeros_like(y), w=w)
    check(out, grads, h, one, torch.zeros_like(y), w)


def test_strides_and_alignment():
    torch = _torch()
    v = gh.verifier()
    B, rows, V, D = 7, 4, 1003, 90
    h, W, y, w = make(B, rows, V, D, 89)
    want = both(v, h, W, y, w=w)
    check(*want, h, W, y, w)

    def laid(t, stride, start, fill=5.0):
        n = t[..., 0].numel()
        flat = torch.full((n * stride + 64,), fill, device="cuda", dtype=t.dtype)
        view = flat[start:start + n * stride].view(*t.shape[:-1], stride)[..., :t.shape[-1]]
        return flat, view
    for hs, h0, ws, gs, g0, vs, v0 in ((90, 0, 96, 90, 0, 96, 0), (91, 1, 104, 93, 3, 90, 2), (96, 8, 128, 96, 4, 104, 8),
                                       (100, 2, 96, 128, 0, 97, 1)):
        _, hv = laid(h, hs, h0, float("nan"))
        hv.copy_(h)
        _, wv = laid(W, ws, 0, float("nan"))
        wv.copy_(W)
        gf, gv = laid(h, gs, g0)
        wf, gw = laid(W, vs, v0)
        out = v.cross_entropy(hv, wv, y)
        assert torch.equal(out["loss"], want[0]["loss"])
        v.cross_entropy_grad(hv, wv, y, out["lse"], grad_loss=w, out={"grad_hidden": gv, "grad_weight": gw})
        assert torch.equal(gv, want[1]["grad_hidden"]) and torch.equal(gw, want[1]["grad_weight"])
        gv.fill_(5.0)
        gw.fill_(5.0)
        assert (gf == 5.0).all() and (wf == 5.0).all()  # nothing beside the rows is written


def test_the_gradient_is_the_losses_slope():
    """Against differences of the call's own losses along a direction: h + e u and h - e u, rounded to bfloat16 as they
    are given, differ by a known d; the slope is grad . d, off by the losses' bounds, the gradient's own bound, the
    third difference (lse's third derivative is below the cube of the largest change of a logit, and a central difference
    leaves a 24th of it) and the distance of the two points' middle from h."""
    torch = _torch()
    v = gh.verifier()
    h, W, y, _ = make(6, 3, 400, 64, 97)
    g = torch.Generator(device="cuda").manual_seed(5)
    u = torch.randn(h.shape, device="cuda", generator=g)
    up, down = (h.float() + 0.02 * u).bfloat16(), (h.float() - 0.02 * u).bfloat16()
    d = up.double() - down.double()
    mid = (up.double() + down.double()) / 2
    lu, ld = (v.cross_entropy(x.contiguous(), W, y)["loss"].double() for x in (up, down))
    lo = cross_entropy_truth(up.double().view(18, 64), W.double(), y.view(18).long())
    grad = v.cross_entropy_grad(h, W, y, v.cross_entropy(h, W, y)["lse"], weight_grad=False)["grad_hidden"].double()
    dz = (d.view(18, 64) @ W.double().T).abs().amax(-1)  # the largest change of a logit
    shift = ((mid - h.double()).view(18, 64) @ W.double().T).abs().amax(-1)
    th = cross_entropy_truth(h.double().view(18, 64), W.double(), y.view(18).long())
    off = 2 * (lo["loss_tol"] + 2.0 ** -24 * lo["loss"].abs()) + dz ** 3 / 24 + dz * shift + \
        (d.view(18, 64).abs() * (th["grad_hidden_tol"] + 2.0 ** -8 * th["grad_hidden"].abs())).sum(-1)
    err = ((lu - ld).view(18) - (grad * d).view(18, 64).sum(-1)).abs()
    assert (err <= off).all()


def test_a_training_step_in_a_graph_and_on_streams():
    """A verify's tokens as labels: loss, both gradients and the distillation of the same rows; captured and replayed on
    other data, and beside it a second graph with a workspace of its own."""
    torch = _torch()
    v = gh.verifier()
    B, K, V, D, T = 12, 3, 3001, 128, 0.9
    K1 = K + 1

    def data(seed):
        h, W, _, w = make(B, K1, V, D, seed)
        W = W.contiguous()
        g = torch.Generator(device="cuda").manual_seed(seed)
        draft = (h.float() @ W.float().T).bfloat16()
        target = (draft.float() + 0.5 * torch.randn(draft.shape, device="cuda", generator=g)).bfloat16()
        u = torch.rand(B, K1, device="cuda", generator=g)
        return [h, W, w, draft, target, u]

    def step(h, W, w, draft, target, u, ws):
        tok = v.sample(draft[:, :K].contiguous(), u[:, :K].contiguous(), temperature=T)["tokens"]
        ver = v.run_draft_logits(target, draft[:, :K].contiguous(), tok, u, T, T)
        lp = v.logprobs(target, ver["out_tokens"], ver["accept_len"], temperature=T, top_n=10)
        out = v.cross_entropy(h, W, ver["out_tokens"], ver["accept_len"], workspace=ws)
        gr = v.cross_entropy_grad(h, W, ver["out_tokens"], out["lse"], ver["accept_len"], grad_loss=w, workspace=ws)
        dis = v.distill(draft, lp["top_logprobs"], lp["top_tokens"], ver["accept_len"], temperature=T, grad_loss=w)
        return ver, lp, out, gr, dis

    def look(x, res):
        from tests.test_gpu_distill import check as check_distill
        ver, lp, out, gr, dis = res
        live = torch.arange(K1, device="cuda")[None] < ver["accept_len"][:, None]
        check(out, gr, x[0], x[1], ver["out_tokens"], x[2], live)
        check_distill(dis, x[3], lp["top_logprobs"], lp["top_tokens"], T, False, x[2], ver["accept_len"].cpu(), "bf16")
    x = data(101)
    ws = v.cross_entropy_workspace(B, K1, V, D)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        res = step(*x, ws)
    s.synchronize()
    look(x, res)
    xs, graphs, results = [data(103), data(107)], [], []
    for y in xs:
        own = v.cross_entropy_workspace(B, K1, V, D)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(step(*y, own))
        graphs.append((graph, own))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed in (109, 113):
        for y, fresh in zip(xs, (data(seed), data(seed + 1))):
            for t, f in zip(y, fresh):
                t.copy_(f)
        torch.cuda.synchronize()
        for (graph, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for y, r in zip(xs, results):
            look(y, r)


def test_two_threads_on_streams_of_their_own():
    torch = _torch()
    import speculative_decoding_verification_14_gb300 as sv
    jobs = [make(20, 4, 4001, 128, s) for s in (127, 131)]
    want = [both(gh.verifier(), h, W, y, w=w) for h, W, y, w in jobs]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            h, W, y, w = jobs[i]
            with sv.Verifier(32, 4, 5000) as v, torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    out, grads = both(v, h, W, y, w=w)
                    torch.cuda.current_stream().synchronize()
                    assert all(torch.equal(out[k], want[i][0][k]) for k in out)
                    assert all(torch.equal(grads[k], want[i][1][k]) for k in grads)
        except BaseException as e:  # handed to the test's own thread
            failed.append(e)
    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not failed, failed


def test_offsets_beyond_32_bits():
    """600 000 rows of 4096: the last ones against the definition; each row's probabilities are one tile wide."""
    torch = _torch()
    v = gh.verifier()
    B, rows, V, D, tail = 20000, 30, 300, 4096, 3
    h, W, y, w = make(tail, rows, V, D, 137)
    big = torch.zeros(B, rows, D, device="cuda", dtype=torch.bfloat16)
    big[-tail:] = h
    yb = torch.full((B, rows), -1, device="cuda", dtype=torch.int32)
    yb[:-tail, ::2] = 5  # packed in front of them
    yb[-tail:] = y
    wb = torch.zeros(B, rows, device="cuda")
    wb[-tail:] = w
    out, grads = both(v, big, W, yb, w=wb)
    part = {k: t[-tail:] for k, t in out.items()}
    check(part, {"grad_hidden": grads["grad_hidden"][-tail:], "grad_weight": grads["grad_weight"]}, h, W, y, w)
    assert (out["lse"][0, ::2] - np.log(V)).abs().max() < 1e-5 and (grads["grad_hidden"][:-tail] == 0).all()
    assert v.error() == (0, 0)


def test_the_first_call_of_a_process_in_a_capture():
    """Kernel attributes and limits are asked for while a stream is captured."""
    import subprocess
    import sys
    code = """
import torch
import speculative_decoding_verification_14_gb300 as sv
torch.cuda.set_device(0)
g = torch.Generator(device="cuda").manual_seed(1)
h = torch.randn(20, 4, 64, device="cuda", generator=g).bfloat16()
W = torch.randn(600, 64, device="cuda", generator=g).bfloat16()
y = torch.randint(0, 600, (20, 4), device="cuda", generator=g, dtype=torch.int32)
z = torch.randn(400, 4, 600, device="cuda", generator=g)
a = torch.randn(400, 4, 7, device="cuda", generator=g)
x = torch.arange(7, device="cuda", dtype=torch.int32).expand(400, 4, 7).contiguous()
v = sv.Verifier(400, 4, 1000)
def step():
    out = v.cross_entropy(h, W, y)
    return [out["loss"], *v.cross_entropy_grad(h, W, y, out["lse"]).values(), *v.distill(z, a, x).values()]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
want = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and v.error() == (0, 0)
print("equal")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stderr
