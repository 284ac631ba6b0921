"""The sampling calls (draw, logit filter, log-probabilities) against their definitions in 64 bits.

Tokens, counts and kept sets are equal wherever the definition's own margin exceeds
sampling_reference.MARGIN.  Probabilities: ex2.approx is off by 2^-22 of its result at most, and the
correction, the scale and the product round once each (2^-24): below 2 * 2^-22; what lies below the
smallest normal float may be flushed.  The kept mass is rounded once (2^-24) from integers."""
import numpy as np
import pytest

from tests import gpu_helpers as gh
from tests.sampling_reference import MARGIN, logprob_truth, row_truth

pytestmark = pytest.mark.gpu

P_RTOL, P_ATOL = 2.0 ** -21, 2.0 ** -126
OFF = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)


def _torch():
    import torch
    return torch


def _tensor(x, dtype):
    torch = _torch()
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()
    return t.bfloat16() if dtype == "bf16" else t


def _f64(t):
    return t.double().cpu().numpy()


def _at(settings, name, b):
    x = settings[name]
    return x[b].item() if hasattr(x, "cpu") else x


def check_rows(lg, settings, u=None, got=None, filtered=None, limit=0.02):
    """Every row of lg [B, rows, V] against the definition; returns rows left out as too near a border."""
    l = _f64(lg)
    B, rows, V = l.shape
    near = 0
    for b in range(B):
        s = {k: _at(settings, k, b) for k in OFF}
        for i in range(rows):
            t = row_truth(l[b, i], s["temperature"], s["top_k"], s["top_p"], s["min_p"],
                          None if u is None else float(u[b, i]))
            where = f"row {b},{i} of V={V} under {s}"
            for out in (got, filtered):
                if out is not None:
                    assert int(out["status"][b, i]) == t["status"], where
                    if t["status"]:
                        assert int(out["kept"][b, i]) == 0
            if t["status"]:
                if got is not None:
                    assert int(got["tokens"][b, i]) == -1 and np.isnan(got["p_token"][b, i])
                    if "probs" in got:
                        assert np.isnan(got["probs"][b, i]).all()
                if filtered is not None:
                    np.testing.assert_array_equal(filtered["logits"][b, i], l[b, i])
                    assert np.isnan(filtered["mass"][b, i])
                continue
            if t["cut_margin"] < MARGIN:
                near += 1
                continue
            if filtered is not None:
                assert int(filtered["kept"][b, i]) == t["kept"], where
                np.testing.assert_array_equal(filtered["logits"][b, i],
                                              np.where(t["keep"], l[b, i], -np.inf), err_msg=where)
                np.testing.assert_allclose(filtered["mass"][b, i], t["mass"], rtol=2.0 ** -24 + 1e-9)
            if got is not None:
                assert int(got["kept"][b, i]) == t["kept"], where
                if "probs" in got:
                    np.testing.assert_array_equal(got["probs"][b, i][~t["keep"]], 0.0, err_msg=where)
                    np.testing.assert_allclose(got["probs"][b, i], t["probs"], rtol=P_RTOL,
                                               atol=P_ATOL, err_msg=where)
                if t["draw_margin"] < MARGIN:
                    near += 1
                    continue
                assert int(got["tokens"][b, i]) == t["token"], where
                np.testing.assert_allclose(got["p_token"][b, i], t["p_token"], rtol=P_RTOL,
                                           atol=P_ATOL)
    assert near <= max(1, limit * B * rows), f"{near} rows at a border"
    return near


def run_all(lg, settings, u=None, cluster=0, probs=True):
    """Draw and filter under a plan; numpy results."""
    torch = _torch()
    v = gh.verifier()
    if u is None:
        g = torch.Generator(device="cuda").manual_seed(lg.shape[-1])
        u = torch.rand(lg.shape[:-1], device="cuda", generator=g)
    if cluster:
        v.set_plan_override(cluster, 0, 0)
    try:
        got = v.sample(lg, u, **settings, probs=probs)
        fil = v.filter_logits(lg, **settings)
        torch.cuda.synchronize()
    finally:
        if cluster:
            v.set_plan_override(0, 0, 0)
    got = {k: t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()
           for k, t in got.items()}
    fil = {k: _f64(t) if t.is_floating_point() else t.cpu().numpy() for k, t in fil.items()}
    return u.cpu().numpy(), got, fil


def rows_of(B, rows, V, seed, scale=2.5):
    return scale * np.random.default_rng(seed).standard_normal((B, rows, V))


SETTINGS = [
    OFF,
    {**OFF, "temperature": 0.6, "top_p": 0.95, "min_p": 0.05},
    {**OFF, "top_k": 1},
    {**OFF, "top_k": 17, "top_p": 0.8},
    {**OFF, "temperature": 1.7, "top_p": 0.9},
    {**OFF, "top_k": 900, "min_p": 0.001},
    {**OFF, "temperature": 0.0, "top_k": 5},
]


@pytest.mark.parametrize("settings", SETTINGS, ids=range(len(SETTINGS)))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 4099, 32000])
def test_shapes(V, dtype, settings):
    lg = _tensor(rows_of(3, 2, V, V), dtype)
    u, got, fil = run_all(lg, settings)
    check_rows(lg, settings, u, got, fil)


@pytest.mark.parametrize("cluster", [1, 2, 3, 8, 16])
@pytest.mark.parametrize("V,dtype", [(20011, "f32"), (20011, "bf16"), (65536, "bf16")])
def test_every_cluster(V, dtype, cluster):
    settings = {**OFF, "top_p": 0.9, "top_k": 4000}
    lg = _tensor(rows_of(2, 1, V, cluster), dtype)
    u, got, fil = run_all(lg, settings, cluster=cluster)
    check_rows(lg, settings, u, got, fil)


@pytest.mark.parametrize("B,V,dtype", [(40, 128256, "bf16"), (24, 151936, "f32"), (200, 4097, "f32")])
def test_batches_of_large_rows(B, V, dtype):
    settings = {**OFF, "top_p": 0.95}
    lg = _tensor(rows_of(B, 1, V, B, 2.0), dtype)
    u, got, fil = run_all(lg, settings)
    check_rows(lg, settings, u, got, fil)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["constant", "two", "few", "narrow", "steep", "signed zeros"])
def test_rows_that_crowd_one_place(kind, dtype):
    """Equal logits by the thousand, and thousands of distinct ones next to each other."""
    rng = np.random.default_rng(5)
    V = 30000
    if kind == "constant":
        x = np.full((4, 1, V), 3.25)
    elif kind == "two":
        x = np.where(rng.random((4, 1, V)) < 0.5, 2.0, 1.0)
    elif kind == "few":
        x = rng.integers(-3, 4, (4, 1, V)).astype(np.float64)
    elif kind == "narrow":
        x = 1.0 + 0.003 * rng.standard_normal((4, 1, V))
    elif kind == "steep":
        x = 1e-3 * rng.standard_normal((4, 1, V))
        x[:, :, 77] = 40.0
    else:
        x = np.where(rng.random((4, 1, V)) < 0.5, 0.0, -0.0)
    lg = _tensor(x, dtype)
    for s in ({**OFF}, {**OFF, "top_p": 0.5}, {**OFF, "top_k": 1500}, {**OFF, "top_k": 12000, "top_p": 0.3},
              {**OFF, "temperature": 30.0, "min_p": 0.95}, {**OFF, "temperature": 0.0}):
        u, got, fil = run_all(lg, s)
        check_rows(lg, s, u, got, fil)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_rows_and_values_that_are_no_logits(dtype):
    torch = _torch()
    V = 5000
    x = rows_of(11, 1, V, 3)
    lowest = float(torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min)
    x[0, 0, 1:] = -np.inf            # one token left
    x[1, 0, :] = -np.inf             # none
    x[2, 0, 100:] = lowest           # masked by the type's lowest value
    x[3, 0, 2500] = np.nan
    x[4, 0, 10] = np.inf
    x[5, 0, ::2] = -np.inf
    x[6, 0, :] = lowest
    x[7, 0, :4990] = -np.inf         # fewer left than top-k
    x[8, 0, V - 1] = np.nan
    x[9, 0, 1:] -= 1e6               # one token carries everything
    lg = _tensor(x, dtype)
    v = gh.verifier()
    v.error()
    for s in SETTINGS:
        u, got, fil = run_all(lg, s)
        check_rows(lg, s, u, got, fil)
    import speculative_decoding_verification_14_gb300 as sv
    assert v.error()[1] == 1 << sv.SV_ERR_NONFINITE


@pytest.mark.parametrize("T", [1e-37, 1e-20, 1e-3, 50.0, 1e20, 3e38])
def test_far_temperatures(T):
    for dtype in ("bf16", "f32"):
        lg = _tensor(rows_of(2, 2, 3001, 8), dtype)
        for s in ({**OFF, "temperature": T}, {**OFF, "temperature": T, "top_p": 0.7, "min_p": 0.3},
                  {**OFF, "temperature": T, "top_k": 40}):
            u, got, fil = run_all(lg, s)
            check_rows(lg, s, u, got, fil)


def test_uniforms_at_the_ends():
    torch = _torch()
    lg = _tensor(np.repeat(rows_of(1, 1, 2000, 9), 6, 0), "f32")
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 2.0 ** -149, 1.0, -0.25, float("nan")], device="cuda")[:, None]
    for s in SETTINGS:
        _, got, _ = run_all(lg, s, u=u)
        assert got["status"][:, 0].tolist() == [0, 0, 0, 7, 7, 7]
        check_rows(lg, s, u.cpu().numpy(), got)
    gh.verifier().error()


def test_settings_of_their_own_for_every_sequence():
    torch = _torch()
    B = 24
    i = torch.arange(B, device="cuda")
    s = {"temperature": (i % 4).float() * 0.5, "top_k": torch.tensor([0, 3, 50], device="cuda",
                                                                    dtype=torch.int32)[i % 3].contiguous(),
         "top_p": torch.tensor([1.0, 0.9, 0.4, 0.99, 2.0], device="cuda")[i % 5].contiguous(),
         "min_p": torch.tensor([0.0, 0.02], device="cuda")[i // 2 % 2].contiguous()}
    s["temperature"][5], s["temperature"][6], s["temperature"][7] = -1.0, float("nan"), float("inf")
    s["top_p"][8], s["top_p"][9] = 0.0, float("nan")
    s["min_p"][10], s["min_p"][11] = 1.0, float("nan")
    lg = _tensor(rows_of(B, 3, 3003, 12), "bf16")
    u, got, fil = run_all(lg, s)
    assert (got["status"][5:12] == 1).all() and (got["status"] == 1).sum() == 21
    check_rows(lg, s, u, got, fil)
    gh.verifier().error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_strides_and_alignment(dtype, shift):
    """Rows inside a wider buffer, starting anywhere; outputs at a draft loop's strides, with what
    lies between them left alone."""
    torch = _torch()
    B, K, V = 5, 3, 1201
    wide = _tensor(rows_of(B, K, V + 61, 4 + shift), dtype)
    lg = wide[:, :, shift:shift + V]
    u = torch.rand(B, K + 1, device="cuda")
    q = torch.full((B, K, V + 8), -3.0, device="cuda")
    draft = torch.full((B, K), -9, dtype=torch.int32, device="cuda")
    s = {**OFF, "top_p": 0.9}
    v = gh.verifier()
    for i in (0, 2):
        out = {"tokens": draft[:, i], "probs": q[:, i, shift:shift + V],
               "status": torch.empty(B, dtype=torch.int32, device="cuda"),
               "kept": torch.empty(B, dtype=torch.int32, device="cuda"),
               "p_token": torch.empty(B, device="cuda")}
        v.sample(lg[:, i], u[:, i], **s, out=out)
        got = {k: t.cpu().numpy()[:, None] for k, t in out.items()}
        check_rows(lg[:, i:i + 1], s, u[:, i:i + 1].cpu().numpy(), got)
    assert (draft[:, 1] == -9).all() and (q[:, 1] == -3.0).all()
    edge = torch.ones_like(q, dtype=torch.bool)
    edge[:, :, shift:shift + V] = False
    assert (q[edge] == -3.0).all()
    # the filter in place, inside the wide buffer
    before, l = wide.clone(), lg.clone()
    fil = v.filter_logits(lg, **s, out={"logits": lg, "kept": torch.empty(B, K, dtype=torch.int32, device="cuda"),
                                        "mass": torch.empty(B, K, device="cuda"),
                                        "status": torch.empty(B, K, dtype=torch.int32, device="cuda")})
    check_rows(l, s, filtered={k: _f64(t) if t.is_floating_point() else t.cpu().numpy() for k, t in fil.items()})
    assert torch.equal(wide[:, :, :shift], before[:, :, :shift])
    assert torch.equal(wide[:, :, shift + V:], before[:, :, shift + V:])


def test_offsets_beyond_32_bits():
    torch = _torch()
    V, step = 2000, (1 << 30) + 8
    buf = torch.empty(2 * step + V, dtype=torch.bfloat16, device="cuda")
    lg = buf.as_strided((3, 1, V), (step, V, 1))
    lg.copy_(_tensor(rows_of(3, 1, V, 2), "bf16"))
    s = {**OFF, "top_p": 0.9}
    l = lg.clone()
    u, got, fil = run_all(lg, s)
    check_rows(l, s, u, got, fil)
    x = torch.tensor(got["tokens"], device="cuda")
    out = gh.verifier().logprobs(lg, x, top_n=3)
    check_logprobs(l, x, None, 1.0, 3, out)


def test_repeated_calls_give_the_same_bits():
    torch = _torch()
    lg = _tensor(rows_of(16, 1, 40000, 1), "f32")
    u = torch.rand(16, 1, device="cuda")
    for s in SETTINGS:
        first = gh.verifier().sample(lg, u, **s, probs=True)
        for cluster in (0, 2, 8):
            gh.verifier().set_plan_override(cluster, 0, 0)
            again = gh.verifier().sample(lg, u, **s, probs=True)
            gh.verifier().set_plan_override(0, 0, 0)
            for k in first:
                assert torch.equal(first[k], again[k]), (s, cluster, k)


# ------------------------------------------------------ log-probabilities -----

# An exponent (l - max) c is off by 2.5 * 2^-24 of itself (the difference, c and the product round),
# which changes a weight by as much times |l - max|/T; ex2.approx adds 2^-22.  The additions of a
# thread's n weights and of the joins round n + 20 times.  Entries far below the maximum weigh
# nothing: 30 bounds the exponent of those that count.  The value itself rounds three times.
def logprob_tol(value, V, threads):
    n = V / threads + 20
    return (30 * 2.5 * 2.0 ** -24 + (n + 8) * 2.0 ** -22 + 4 * 2.0 ** -24 * (1 + np.abs(value)))


def check_logprobs(lg, x, n_live, T, top_n, out):
    l = _f64(lg)
    if l.ndim == 2:
        l, x = l[:, None], x[:, None]
    B, rows, V = l.shape
    o = {k: t.cpu().numpy().reshape((B, rows) + ((top_n,) if k.startswith("top") else ()))
         for k, t in out.items()}
    x = x.cpu().numpy()
    for b in range(B):
        for i in range(rows):
            where = f"row {b},{i} V={V}"
            live = n_live is None or i < int(n_live[b])
            t = logprob_truth(l[b, i], int(x[b, i]), T, top_n) if live else {"status": 0}
            assert o["status"][b, i] == t["status"], where
            if not live or t["status"]:
                assert np.isnan(o["logprob"][b, i]) and o["rank"][b, i] == 0
                if top_n:
                    assert np.isnan(o["top_logprobs"][b, i]).all() and (o["top_tokens"][b, i] == -1).all()
                continue
            assert o["rank"][b, i] == t["rank"], where
            np.testing.assert_allclose(o["logprob"][b, i], t["logprob"], rtol=0,
                                       atol=logprob_tol(t["logprob"] if np.isfinite(t["logprob"]) else 0, V, 256))
            if top_n:
                np.testing.assert_array_equal(o["top_tokens"][b, i], t["top_tokens"], err_msg=where)
                fin = t["top_tokens"] >= 0
                assert np.isnan(o["top_logprobs"][b, i][~fin]).all()
                assert (np.abs(o["top_logprobs"][b, i][fin] - t["top_logprobs"][fin])
                        <= logprob_tol(t["top_logprobs"][fin], V, 256)).all(), where


@pytest.mark.parametrize("top_n", [0, 1, 5, 32])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 3, 40, 1000, 4099, 32000])
def test_logprobs(V, dtype, top_n):
    torch = _torch()
    B, rows, T = 6, 3, 0.8
    lg = _tensor(rows_of(B, rows, V, V + top_n), dtype)
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randint(0, V, (B, rows), device="cuda", generator=g, dtype=torch.int32)
    n = torch.tensor([0, 1, 2, 3, 3, 2], device="cuda", dtype=torch.int32)
    x = torch.where(torch.arange(rows, device="cuda")[None] < n[:, None], x, -1).to(torch.int32)
    x[4, 0] = V
    x[5, 1] = -1
    out = gh.verifier().logprobs(lg, x, n, temperature=T, top_n=top_n)
    check_logprobs(lg, x, n, T, top_n, out)
    gh.verifier().error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logprobs_of_rows_with_ties_and_masks(dtype):
    torch = _torch()
    V = 20000
    rng = np.random.default_rng(0)
    x = rows_of(9, 1, V, 1)
    x[0] = 1.5                                        # every entry equal
    x[1] = rng.integers(0, 3, V)                      # thousands of the largest
    x[2, 0, 7:] = -np.inf                             # fewer than asked for
    x[3, 0, :] = -np.inf
    x[4, 0, 19999] = np.nan
    x[5, 0, 0] = np.inf
    x[6, 0, 10:] = float(torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min)
    x[7] = np.sort(x[7], axis=-1)                     # the largest in one thread's and CTA's reach
    x[8] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    lg = _tensor(x, dtype)
    t = torch.tensor([[5], [9], [3], [0], [0], [0], [4], [V - 1], [11]], device="cuda", dtype=torch.int32)
    for cluster in (0, 1, 2, 16):
        gh.verifier().set_plan_override(cluster, 0, 0)
        try:
            for top_n in (1, 20, 32):
                check_logprobs(lg, t, None, 1.0, top_n, gh.verifier().logprobs(lg, t, top_n=top_n))
        finally:
            gh.verifier().set_plan_override(0, 0, 0)
    t[2, 0] = 12                                      # a token of probability 0
    check_logprobs(lg, t, None, 1.0, 8, gh.verifier().logprobs(lg, t, top_n=8))
    gh.verifier().error()


def test_logprobs_leave_rows_behind_the_last_unread():
    torch = _torch()
    lg = _tensor(rows_of(4, 4, 3000, 0), "bf16")
    n = torch.tensor([1, 2, 4, 0], device="cuda", dtype=torch.int32)
    for b in range(4):
        lg[b, int(n[b]):] = float("nan")
    x = torch.full((4, 4), 17, device="cuda", dtype=torch.int32)
    gh.verifier().error()
    out = gh.verifier().logprobs(lg, x, n, top_n=4)
    assert (out["status"] == 0).all() and gh.verifier().error() == (0, 0)
    check_logprobs(lg.nan_to_num(0.0), x, n, 1.0, 4, out)
