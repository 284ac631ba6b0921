"""A head of one token: its row's distance to the next, which there is none of, does not matter."""
import pytest

from tests import gpu_helpers as gh

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [1, 9, 90, 1001])
def test_any_depth(D):
    """loss 0, lse the logit, d = 0: both gradients 0."""
    import torch
    v = gh.verifier()
    g = torch.Generator(device="cuda").manual_seed(D)
    h = torch.randn(5, 3, D, device="cuda", generator=g).bfloat16()
    W = torch.randn(1, D, device="cuda", generator=g).bfloat16()
    y = torch.zeros(5, 3, device="cuda", dtype=torch.int32)
    out = v.cross_entropy(h, W, y)
    z = (h.double() * W.double()[0]).sum(-1)
    size = (h.double() * W.double()[0]).abs().sum(-1)
    # float32 sums of exact products, which the tensor cores may cut
    assert ((out["lse"].double() - z).abs() <= (D / 16 + 17) * 2.0 ** -23 * size + 2.0 ** -24 * z.abs()).all()
    assert (out["loss"] == 0).all() and (out["status"] == 0).all()
    got = v.cross_entropy_grad(h, W, y, out["lse"], loss=out["loss"])
    assert all((t == 0).all() for t in got.values())
    # the gradients of an lse that is half a unit off in its last place
    got = v.cross_entropy_grad(h, W, y, out["lse"])
    assert all((t.abs() <= 1e-4).all() for t in got.values())


def test_a_gradient_far_from_a_next_row():
    """The longest stride that is taken: the copy engine's own end before it."""
    import torch
    import speculative_decoding_verification_14_gb300 as sv
    v = gh.verifier()
    h = torch.ones(2, 16, device="cuda").bfloat16()
    W = torch.ones(1, 16, device="cuda").bfloat16()
    y = torch.zeros(2, device="cuda", dtype=torch.int32)
    out = v.cross_entropy(h, W, y)
    ws = v.cross_entropy_workspace(2, 1, 1, 16)
    beside = torch.full((3, 16), 7.0, device="cuda").bfloat16()
    for stride in (16, (1 << 39) - 8, 1 << 39, (1 << 40) - 8):
        beside[1] = 7.0
        assert sv.spec_cross_entropy_grad(v.ctx, h.data_ptr(), 1, 16, W.data_ptr(), 16, y.data_ptr(), None, out["lse"].data_ptr(),
                                          None, 2, 1, 1, 16, None, 0, beside[1].data_ptr(), stride, None, ws.data_ptr(),
                                          ws.numel()) == sv.SV_OK, stride
        torch.cuda.synchronize()
        assert (beside[1] == 0).all() and (beside[0] == 7).all() and (beside[2] == 7).all()
