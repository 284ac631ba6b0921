"""Memory that a call allocates belongs to the stream it launches on: torch hands out what was freed on a stream to
that stream's next allocation, ordered behind it and behind nothing else."""
import contextlib

import pytest


def calls(torch, device):
    """Every method that allocates, as name and call of (verifier, stream)."""
    B, K, V, n, D = 2, 3, 64, 4, 8
    f = lambda *s: torch.zeros(*s, device=device)
    i = lambda *s: torch.zeros(*s, device=device, dtype=torch.int32)
    lg, q, tok, u = f(B, K + 1, V), f(B, K, V) + 1.0 / V, i(B, K), f(B, K + 1) + 0.5
    h, W, y, lse = f(B, K + 1, D).bfloat16(), f(V, D).bfloat16(), i(B, K + 1), f(B, K + 1) + 4.0
    a, x = f(B, K + 1, n), torch.arange(n, device=device, dtype=torch.int32).expand(B, K + 1, n).contiguous()
    offsets = torch.tensor([0, K + 1, 2 * (K + 1)], device=device, dtype=torch.int32)
    return {
        "run": lambda v, s: v.run(lg, q, tok, u, 1.0, stats=True, stream=s),
        "run_greedy": lambda v, s: v.run_greedy(lg, tok, argmax=True, stream=s),
        "run_ragged": lambda v, s: v.run_ragged(lg.view(-1, V), q.view(-1, V), tok.view(-1), u.view(-1), offsets, K, 1.0,
                                                stats=True, stream=s),
        "run_truncated": lambda v, s: v.run_truncated(lg, q, tok, u, 1.0, 0.9, 0.0, stats=True, stream=s),
        "run_draft_logits": lambda v, s: v.run_draft_logits(lg, lg[:, :K].contiguous(), tok, u, 1.0, 1.0, stats=True, stream=s),
        "sample": lambda v, s: v.sample(lg, u, probs=True, stream=s),
        "filter_logits": lambda v, s: v.filter_logits(lg, top_k=5, stream=s),
        "logprobs": lambda v, s: v.logprobs(lg, y, top_n=n, stream=s),
        "distill": lambda v, s: v.distill(lg, a, x, stream=s),
        "cross_entropy": lambda v, s: v.cross_entropy(h, W, y, stream=s),
        "cross_entropy_grad": lambda v, s: v.cross_entropy_grad(h, W, y, lse, status=True, stream=s),
    }


NAMES = ("run", "run_greedy", "run_ragged", "run_truncated", "run_draft_logits", "sample", "filter_logits", "logprobs",
         "distill", "cross_entropy", "cross_entropy_grad")


@pytest.mark.parametrize("stream", [0, 0x5150])
@pytest.mark.parametrize("name", NAMES)
def test_allocations_are_made_under_the_stream(name, stream, monkeypatch):
    """On the host, a library and streams that only take notes."""
    import torch
    import speculative_decoding_verification_14_gb300 as sv

    class Library:
        def __getattr__(self, _):
            return lambda *a: sv.SV_OK
    inside, made, bare = [], [], torch.empty

    @contextlib.contextmanager
    def under(s):
        inside.append(s)
        yield
        inside.pop()

    def empty(*shape, device=None, **kw):
        made.append(inside[-1] if inside else None)
        return bare(*shape, **kw)
    job = calls(torch, "cpu")[name]
    monkeypatch.setattr(sv, "library", Library)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda p, device=None: ("given", p))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("given", 0))
    v = object.__new__(sv.Verifier)
    v.device, v.ctx = -1, None
    out = job(v, stream)
    assert out and len(made) >= len(out) and all(s == ("given", stream) for s in made), made


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_outputs_lie_in_the_streams_memory(name):
    """As torch's allocator says, and with the answers of a call on the current stream."""
    import torch
    from tests import gpu_helpers as gh
    v = gh.verifier()
    job = calls(torch, "cuda")[name]
    want = job(v, None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = job(v, s.cuda_stream)
    s.synchronize()
    segments = torch.cuda.memory_snapshot()
    default = job(v, 0)
    torch.cuda.synchronize()
    whole = set(want) if name in ("distill", "cross_entropy", "cross_entropy_grad") else {"status"}  # no place left unwritten
    for k, t in got.items():
        owner = [g["stream"] for g in segments if g["address"] <= t.data_ptr() < g["address"] + g["total_size"]]
        assert owner == [s.cuda_stream], k
        assert k not in whole or torch.equal(t, want[k]) and torch.equal(default[k], want[k]), k


@pytest.mark.gpu
@pytest.mark.parametrize("named", [False, True])
@pytest.mark.parametrize("B,rows,lengths", [(6, 3, False), (9001, 1, False), (700, 4, True)])
def test_captured_with_losses_and_without_a_workspace(B, rows, lengths, named):
    """A training step of loss, gradients given the losses, and no memory of the caller's, captured on a stream that the
    calls are told of or find current; replayed on other data, with the answers of calls on the default stream."""
    import torch
    from tests import gpu_helpers as gh
    v = gh.verifier()
    V, D = 300, 24

    def data(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        W = torch.randn(V, D, device="cuda", generator=g).bfloat16()
        y = torch.randint(-1, V, (B, rows), device="cuda", generator=g, dtype=torch.int32)
        h = (torch.randn(B, rows, D, device="cuda", generator=g) + 0.5 * W[y.clamp(min=0).long()].float()).bfloat16()
        return [h, W, y, torch.randint(0, rows + 1, (B,), device="cuda", generator=g, dtype=torch.int32),
                torch.rand(B, rows, device="cuda", generator=g)]

    def step(x, **kw):
        h, W, y, lens, w = x
        lens = lens if lengths else None
        out = v.cross_entropy(h, W, y, lens, **kw)
        return {**out, **v.cross_entropy_grad(h, W, y, out["lse"], lens, grad_loss=w, loss=out["loss"], **kw)}
    x = data(1)
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step(x, **({"stream": s.cuda_stream} if named else {}))
    for seed in (2, 3):
        for t, f in zip(x, data(seed)):
            t.copy_(f)
        graph.replay()
        want = step(x)
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want) and (want["status"] == 0).all()
