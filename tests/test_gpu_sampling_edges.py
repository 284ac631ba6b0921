"""The sampling calls at the edges of what they are documented to take."""
import numpy as np
import pytest

from tests import gpu_helpers as gh
from tests.test_gpu_sampling import OFF, SETTINGS, _tensor, check_logprobs, check_rows, rows_of

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


def general_rows(lg, settings, u=None, limit=0.02):
    """How many rows of a draw, and of a filter, go the general way; their answers are checked."""
    import torch
    v = gh.verifier()
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    u = torch.rand(lg.shape[:-1], device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)) \
        if u is None else u
    try:
        v.set_sample_telemetry(n[0])
        got = v.sample(lg, u, **settings, probs=True)
        v.set_sample_telemetry(n[1])
        fil = v.filter_logits(lg, **settings)
    finally:
        v.set_sample_telemetry(None)
    v.sample(lg, u, **settings)  # not counted
    check_rows(lg, settings, u.cpu().numpy(), {k: t.cpu().numpy() for k, t in got.items()},
               {k: t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy() for k, t in fil.items()}, limit)
    return n.tolist()


def shaped(kind, B, V, seed):
    x = rows_of(B, 1, V, seed, 1.0)
    if kind == "normal":
        return 2.5 * x
    if kind == "peaked":
        return 3.0 * x + 8.0 * (np.random.default_rng(seed).random(x.shape) < 0.01)
    if kind == "zipf":
        return 2.0 * x - 1.1 * np.log(np.arange(1, V + 1))
    if kind == "masked":
        return np.where(np.random.default_rng(seed).random(x.shape) < 0.9, -np.inf, 2.5 * x)
    lowest = -3.3895313892515355e38  # bfloat16's
    return np.where(np.random.default_rng(seed).random(x.shape) < 0.9, lowest, 2.5 * x)


QUICK = [OFF, {**OFF, "top_k": 50, "top_p": 0.95}, {**OFF, "temperature": 0.6, "top_p": 0.95, "min_p": 0.05}]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["normal", "peaked", "zipf", "masked", "lowest"])
def test_ordinary_rows_are_settled_by_counting(kind, dtype):
    B, V = 8, 20011
    lg = _tensor(shaped(kind, B, V, 3), dtype)
    for s in QUICK:
        assert general_rows(lg, s) == [0, 0], s


def test_rows_that_go_the_general_way():
    B, V = 4, 4000
    x = shaped("normal", B, V, 3)
    assert general_rows(_tensor(x + 200.0, "bf16"), OFF) == [B, B]
    assert general_rows(_tensor(x + 200.0, "f32"), OFF) == [B, B]
    assert general_rows(_tensor(x, "f32"), {**OFF, "temperature": 0.0}) == [B, B]
    assert general_rows(_tensor(x, "bf16"), {**OFF, "temperature": 0.0}) == [0, 0]
    assert general_rows(_tensor(1.0 + 1e-3 * x, "f32"), {**OFF, "top_p": 0.5}) == [B, B]
    x[2, 0, 7] = np.nan
    assert general_rows(_tensor(x, "f32"), OFF) == [1, 1]
    gh.verifier().error()


def test_telemetry_refusals():
    import torch
    import speculative_decoding_verification_14_gb300 as sv
    v = gh.verifier()
    assert sv.spec_sample_set_telemetry(v.ctx, 2) == sv.SV_ERR_INVALID_ARG
    for bad in (torch.zeros(1), torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32)):
        with pytest.raises((TypeError, ValueError)):
            v.set_sample_telemetry(bad)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1.2e-38, 1e-30, 1e-10, 1e-5, 1e-4, 3e-4, 1e-3, 3e-3, 0.01, 0.03, 0.1])
def test_low_temperatures(T, dtype):
    """A row's mass is that of its largest few entries, however little a logit half a place below weighs."""
    import torch
    x = rows_of(16, 1, 3000, 5)
    x[8:] *= 0.1
    lg = _tensor(x, dtype)
    for s in ({"top_p": 0.9}, {"top_p": 0.3}, {"top_p": 0.999, "top_k": 40}, {"top_p": 0.5, "min_p": 0.2}, {}):
        s = {**OFF, "temperature": T, **s}
        general_rows(lg, s, torch.rand(16, 1, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)))


@pytest.mark.parametrize("zeros", [0, 4])
def test_a_few_zeros_do_not_narrow_the_stretches(zeros):
    """Half of each row's mass in two entries, one of them at its place's lower end: the places' sums are
    off by up to 0.8 % of the row (2^-5 of a quarter), within four deviations (4 * 2^-4 / sqrt(12) of
    the quarter), and the entries around the cut weigh a few 2^-14 each.  A few logits below the counted
    magnitudes, as a padded vocabulary's, change nothing."""
    import torch
    B, V = 32, 4096
    rng = np.random.default_rng(8)
    x = rng.standard_normal((B, 1, V))
    x[:, :, 11], x[:, :, 12] = 8.0, 8.07
    if zeros:
        x[:, :, -zeros:] = 0.0
    lg = _tensor(x, "f32")
    p = torch.tensor(rng.uniform(0.6, 0.9, B).astype(np.float32), device="cuda")
    assert general_rows(lg, {**OFF, "top_p": p}) == [0, 0]


def test_deviations_beyond_what_a_float_holds():
    """At T = 1e-30 the square of a place's width over T is no float."""
    lg = _tensor(rows_of(4, 1, 3000, 5), "f32")
    assert general_rows(lg, {**OFF, "temperature": 1e-30, "top_p": 0.9}) == [0, 0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1e29, 3e36, 1e38, 3.4e38])
def test_logits_further_apart_than_a_float_holds(T, dtype):
    """Finite logits whose difference is none, at temperatures that weigh it.  The weights of row 3's
    ordinary logits are all 1 there, and 0.7 of 2000 end with an entry: of the 12 rows its two are at a
    border, which is the limit."""
    import torch
    rng = np.random.default_rng(4)
    x = 3.3e38 * rng.uniform(-1, 1, (6, 2, 2000))
    x[2] = np.where(rng.random((2, 2000)) < 0.5, 3.3e38, -3.3e38)
    x[3] = rows_of(1, 2, 2000, 3)[0]
    x[4, :, 5] = -np.inf
    lg = _tensor(x, dtype)
    for s in ({}, {"top_p": 0.7}, {"min_p": 0.4}, {"top_k": 30}, {"top_k": 700, "top_p": 0.5, "min_p": 0.2}):
        general_rows(lg, {**OFF, "temperature": T, **s}, torch.rand(6, 2, device="cuda"), 2 / 12)
    t = torch.randint(0, 2000, (6, 2), device="cuda", dtype=torch.int32)
    check_logprobs(lg, t, None, T, 5, gh.verifier().logprobs(lg, t, temperature=T, top_n=5))


def test_rows_out_between_the_rows_in():
    """Logits, truncated logits and probabilities side by side in one buffer: apart, though the stretches they
    lie in are not.  One entry less apart is refused."""
    import torch
    import speculative_decoding_verification_14_gb300 as sv
    B, rows, V, wide = 5, 3, 700, 2200
    buf = torch.full((B, rows, wide), -3.0, device="cuda")
    lg, cut, q = buf[:, :, :V], buf[:, :, V:2 * V], buf[:, :, 2 * V:3 * V]
    lg.copy_(_tensor(rows_of(B, rows, V, 4), "f32"))
    l, s = lg.clone(), {**OFF, "top_p": 0.9}
    u = torch.rand(B, rows, device="cuda")
    v = gh.verifier()
    want, cut_want = v.sample(l, u, **s, probs=True), v.filter_logits(l, **s)
    tokens = torch.empty(B, rows, dtype=torch.int32, device="cuda")
    v.sample(lg, u, **s, out={"tokens": tokens, "probs": q})
    v.filter_logits(lg, **s, out={"logits": cut})
    assert torch.equal(q, want["probs"]) and torch.equal(tokens, want["tokens"]) and torch.equal(cut, cut_want["logits"])
    assert torch.equal(lg, l) and (buf[:, :, 3 * V:] == -3.0).all()
    for off in (V - 1, wide - V + 1):  # the end of its own row, the start of the next
        near = buf.as_strided((B - 1, rows, V), (rows * wide, wide, 1), off)
        for call in (lambda: v.sample(lg[:-1], u[:-1], **s, out={"tokens": tokens[:-1], "probs": near}),
                     lambda: v.filter_logits(lg[:-1], **s, out={"logits": near})):
            with pytest.raises(sv.SpecVerifyError):
                call()
