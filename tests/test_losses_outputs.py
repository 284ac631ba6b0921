"""Which outputs a losses' call writes: those of its ``out``, or without one those its flags ask for."""
import itertools

import pytest


@pytest.fixture
def seen(monkeypatch):
    """A verifier on the host whose library notes its arguments."""
    import torch
    import speculative_decoding_verification_14_gb300 as sv
    calls = {}

    class Library:
        def __getattr__(self, name):
            return lambda *a: calls.__setitem__(name, a) or sv.SV_OK
    bare = torch.empty
    monkeypatch.setattr(sv, "library", Library)
    monkeypatch.setattr(torch, "empty", lambda *s, device=None, **kw: bare(*s, **kw))
    v = object.__new__(sv.Verifier)
    v.device, v.ctx = -1, None
    return v, calls


@pytest.mark.parametrize("held", [c for n in range(1, 4) for c in itertools.combinations(("loss", "grad_logits", "status"), n)])
@pytest.mark.parametrize("flag", [False, True])
def test_distill(seen, held, flag):
    import torch
    v, calls = seen
    lg, a, x = torch.zeros(2, 3, 8), torch.zeros(2, 3, 4), torch.zeros(2, 3, 4, dtype=torch.int32)
    new = {"loss": torch.zeros(2, 3), "grad_logits": torch.zeros(2, 3, 8), "status": torch.zeros(2, 3, dtype=torch.int32)}
    place = {"loss": 14, "grad_logits": 15, "status": 17}
    out = {k: new[k] for k in held}
    assert v.distill(lg, a, x, loss=flag, grad=flag, status=flag, out=out, stream=0) is out
    for k in new:
        assert calls["spec_distill_run"][place[k]] == (new[k].data_ptr() if k in held else None)


@pytest.mark.parametrize("held", [c for n in range(1, 4) for c in itertools.combinations(("grad_hidden", "grad_weight", "status"), n)])
@pytest.mark.parametrize("flag", [False, True])
def test_cross_entropy_grad(seen, held, flag):
    import torch
    v, calls = seen
    h, W = torch.zeros(2, 3, 8).bfloat16(), torch.zeros(5, 8).bfloat16()
    y, lse, ws = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3), torch.zeros(8, dtype=torch.uint8)
    new = {"grad_hidden": torch.zeros_like(h), "grad_weight": torch.zeros_like(W), "status": torch.zeros_like(y)}
    place = {"grad_hidden": 15, "grad_weight": 17, "status": 19}
    out = {k: new[k] for k in held}
    assert v.cross_entropy_grad(h, W, y, lse, hidden_grad=flag, weight_grad=flag, status=flag, out=out, workspace=ws,
                                stream=0) is out
    for k in new:
        assert calls["spec_cross_entropy_grad_of_loss"][place[k]] == (new[k].data_ptr() if k in held else None)
