"""The sampling calls at the edges of what they are documented to take."""
import numpy as np
import pytest

from tests import gpu_helpers as gh
from tests.test_gpu_sampling import OFF, SETTINGS, _tensor, check_rows, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_uniform_of_minus_zero_is_zero(dtype):
    """On rows of every way through the kernel: ordinary ones, ones beyond the counted logits, and
    ones whose entries crowd one place."""
    import torch
    V = 3000
    x = rows_of(3, 2, V, 14)
    x[1] += 200.0
    x[2] = np.where(np.arange(V) % 2, 1.0, 2.0)
    lg = _tensor(x, dtype)
    u = torch.zeros(3, 2, device="cuda")
    for s in SETTINGS:
        want = gh.verifier().sample(lg, u, **s, probs=True)
        got = gh.verifier().sample(lg, -u, **s, probs=True)
        assert all(torch.equal(got[k], want[k]) for k in want)
        check_rows(lg, s, (-u).cpu().numpy(), {k: t.cpu().numpy() for k, t in got.items()})
