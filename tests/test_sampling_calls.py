"""Sampling calls: refusals, the planner, and the definition the GPU tests compare with."""
import ctypes
import itertools

import numpy as np
import pytest

import oracle
from tests.sampling_reference import logprob_truth, row_truth


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_14_gb300 import build
    build.build()
    import speculative_decoding_verification_14_gb300 as pkg
    return pkg


def test_worked_examples():
    l = np.log([.5, .3, .15, .05])
    assert row_truth(l, 1.0, top_p=.9)["keep"].tolist() == [True, True, True, False]
    assert row_truth(l, 1.0, min_p=.35)["keep"].tolist() == [True, True, False, False]
    assert row_truth(l, 1.0, top_k=1)["keep"].tolist() == [True, False, False, False]
    # ties at a border stay together
    assert row_truth([1., 2., 1., 1.], 1.0, top_k=2)["kept"] == 4
    assert row_truth([1., 2., 2., 1.], 1.0, top_k=2)["kept"] == 2
    # by descending logit, then ascending id: cut points .5, .8, .95
    l = np.log([.15, .5, .05, .3])
    assert [row_truth(l, 1.0, u=u)["token"] for u in (0.0, .49, .51, .81, .96)] == [1, 1, 3, 0, 2]
    assert row_truth([2., 5., 5., 1.], 0.0, u=.9)["token"] == 1
    t = logprob_truth(np.log([.25, .5, .25]), 2, 1.0, 4)
    assert abs(t["logprob"] - np.log(.25)) < 1e-12 and t["rank"] == 2
    assert t["top_tokens"].tolist() == [1, 0, 2, -1]


@pytest.mark.parametrize("top_p,min_p", [(.9, 0.), (1., .05), (.8, .02)])
def test_the_kept_distribution_is_the_truncated_verifys(top_p, min_p):
    """K = 0 draws of the truncated verify's oracle, at uniforms between all cut points by ascending id."""
    rng = np.random.default_rng(3)
    l = (2 * rng.standard_normal(60)).astype(np.float32)
    t = row_truth(l, .7, top_p=top_p, min_p=min_p)
    cut = np.cumsum(t["probs"])
    mid = (np.r_[0.0, cut[:-1]] + cut)[t["keep"]] / 2
    M = len(mid)
    out = oracle.verify_truncated(np.broadcast_to(l, (M, 1, 60)), "f32", np.zeros((M, 0, 60), np.float32),
                                  np.zeros((M, 0), np.int32), mid.astype(np.float32)[:, None], .7, top_p, min_p)
    assert out["out_tokens"][:, 0].tolist() == np.flatnonzero(t["keep"]).tolist()


@pytest.mark.parametrize("op", ["sample", "logprobs"])
@pytest.mark.parametrize("B,rows,V,dtype", list(itertools.product(
    [1, 3, 64, 256, 5000], [1, 5, 33], [1, 7, 4099, 32000, 128256, 151936, 1 << 31], [0, 1])))
def test_plans(sv, op, B, rows, V, dtype):
    rc, p = getattr(sv, f"spec_{op}_plan_for")(152, 16, B, rows, V, dtype)
    assert rc == sv.SV_OK
    C, s = p["cluster"], p["slice"]
    assert C in (1, 2, 4, 8, 16) and p["grid"] == B * rows * C
    assert s % 8 == 0 and s * C >= V and s * (C - 1) < V + 8 * C
    for c in (1, 3, 16):
        rc, p = getattr(sv, f"spec_{op}_plan_for")(152, 16, B, rows, V, dtype, c)
        assert rc == sv.SV_OK and p["cluster"] == c and p["slice"] * c >= V


@pytest.mark.parametrize("op", ["sample", "logprobs"])
def test_plan_refusals(sv, op):
    f = getattr(sv, f"spec_{op}_plan_for")
    for bad in ((0, 16, 1, 1, 10, 0), (152, 0, 1, 1, 10, 0), (152, 16, 0, 1, 10, 0),
                (152, 16, 1, 0, 10, 0), (152, 16, 1, 34, 10, 0), (152, 16, 1, 1, 0, 0),
                (152, 16, 1, 1, (1 << 31) + 1, 0), (152, 16, 1, 1, 10, 2), (152, 16, 1, 1, 10, 0, 17),
                (152, 16, 1, 1, 10, 0, -1)):
        assert f(*bad)[0] == sv.SV_ERR_INVALID_ARG, bad
    assert f(152, 8, 1, 1, 10, 0, 16)[0] == sv.SV_ERR_UNSUPPORTED
    assert getattr(sv.library(), f"spec_{op}_get_plan")(None, 1, 1, 10, 0, ctypes.byref(sv.sv_plan())) == \
        sv.SV_ERR_INVALID_ARG


def test_null_context(sv):
    s = sv.sv_sampling(temperature=1.0, top_p=1.0)
    assert sv.spec_sample_run(None, 16, 0, 10, 16, 1, 1, 1, 10, s, 16, 1) == sv.SV_ERR_INVALID_ARG
    assert sv.spec_filter_run(None, 16, 0, 10, 1, 1, 10, s, 16, 10) == sv.SV_ERR_INVALID_ARG
    assert sv.spec_logprobs_run(None, 16, 0, 10, 16, 16, 1, 1, 10, 1.0, 0, 16) == sv.SV_ERR_INVALID_ARG


@pytest.mark.gpu
def test_refusals_launch_nothing(sv):
    """Every argument that is checked, one at a time out of a call that would be taken."""
    import torch
    B, rows, V = 2, 3, 64
    lg = torch.zeros(B, rows, V, device="cuda")
    u = torch.zeros(B, rows, device="cuda")
    tok = torch.full((B, rows), -7, device="cuda", dtype=torch.int32)
    out = torch.full((B, rows, V), -7.0, device="cuda")
    ints = torch.full((B * rows,), -7, device="cuda", dtype=torch.int32)
    fl = torch.full((B * rows,), -7.0, device="cuda")
    with sv.Verifier(4, 4, 100) as v:
        good = sv.sv_sampling(temperature=1.0, top_p=1.0)

        def settings(**kw):
            return sv.sv_sampling(**{"temperature": 1.0, "top_p": 1.0, **kw})

        sample = dict(ctx=v.ctx, logits_ptr=lg.data_ptr(), dtype=0, logits_stride=V, uniforms_ptr=u.data_ptr(),
                      uniforms_stride=1, B=B, rows_per_seq=rows, V=V, settings=good, tokens_ptr=tok.data_ptr(),
                      tokens_stride=1, probs_ptr=out.data_ptr(), probs_stride=V, p_token_ptr=fl.data_ptr(),
                      kept_ptr=ints.data_ptr(), status_ptr=ints.data_ptr())
        shared = [dict(logits_ptr=None), dict(logits_ptr=lg.data_ptr() + 2), dict(dtype=2),
                  dict(logits_stride=V - 1), dict(logits_stride=1 << 41), dict(B=0), dict(B=5),
                  dict(rows_per_seq=0), dict(rows_per_seq=6), dict(V=0), dict(V=101),
                  dict(status_ptr=ints.data_ptr() + 1)]
        bad_settings = [dict(settings=settings(**kw)) for kw in (
            dict(temperature=-1.0), dict(temperature=float("nan")), dict(temperature=float("inf")),
            dict(temperature=1e-40), dict(top_p=0.0), dict(top_p=float("nan")), dict(min_p=1.0),
            dict(min_p=float("nan")), dict(temperatures=fl.data_ptr() + 1), dict(top_ks=fl.data_ptr() + 2),
            dict(top_ps=fl.data_ptr() + 3), dict(min_ps=fl.data_ptr() + 1))]
        for bad in shared + bad_settings + [
                dict(uniforms_ptr=None), dict(uniforms_ptr=u.data_ptr() + 1), dict(uniforms_stride=0),
                dict(tokens_ptr=None), dict(tokens_stride=0), dict(tokens_ptr=tok.data_ptr() + 1),
                dict(probs_stride=V - 1), dict(probs_ptr=out.data_ptr() + 1), dict(probs_ptr=lg.data_ptr()),
                dict(probs_ptr=lg.data_ptr() + 4 * V), dict(kept_ptr=ints.data_ptr() + 1),
                dict(p_token_ptr=fl.data_ptr() + 1)]:
            assert sv.spec_sample_run(**{**sample, **bad}) == sv.SV_ERR_INVALID_ARG, bad
        filt = {k: sample[k] for k in ("ctx", "logits_ptr", "dtype", "logits_stride", "B", "rows_per_seq", "V",
                                       "settings", "kept_ptr", "status_ptr")}
        filt.update(out_ptr=out.data_ptr(), out_stride=V, mass_ptr=fl.data_ptr())
        for bad in shared + bad_settings + [
                dict(out_ptr=None), dict(out_ptr=out.data_ptr() + 1), dict(out_stride=V - 1),
                dict(mass_ptr=fl.data_ptr() + 1), dict(out_ptr=lg.data_ptr() + 4),
                dict(out_ptr=lg.data_ptr(), out_stride=V + 1), dict(out_ptr=lg.data_ptr() - 4)]:
            assert sv.spec_filter_run(**{**filt, **bad}) == sv.SV_ERR_INVALID_ARG, bad
        lp = {k: sample[k] for k in ("ctx", "logits_ptr", "dtype", "logits_stride", "tokens_ptr", "B",
                                     "rows_per_seq", "V", "status_ptr")}
        lp.update(accept_len_ptr=None, T=1.0, top_n=4, logprob_ptr=fl.data_ptr(), rank_ptr=ints.data_ptr(),
                  top_logprobs_ptr=out.data_ptr(), top_tokens_ptr=out.data_ptr())
        for bad in shared + [dict(tokens_ptr=None), dict(T=0.0), dict(T=float("nan")), dict(T=float("inf")),
                             dict(top_n=-1), dict(top_n=33), dict(top_logprobs_ptr=None),
                             dict(top_tokens_ptr=None), dict(logprob_ptr=None), dict(rank_ptr=ints.data_ptr() + 2),
                             dict(accept_len_ptr=ints.data_ptr() + 1)]:
            assert sv.spec_logprobs_run(**{**lp, **bad}) == sv.SV_ERR_INVALID_ARG, bad
        torch.cuda.synchronize()
        assert (tok == -7).all() and (out == -7.0).all() and (ints == -7).all() and (fl == -7.0).all()
        assert v.error() == (0, 0)


@pytest.mark.gpu
def test_the_wrapper_refuses_what_the_library_cannot_see(sv):
    import torch
    with sv.Verifier(4, 4, 100) as v:
        lg, u = torch.zeros(2, 3, 64, device="cuda"), torch.zeros(2, 3, device="cuda")
        for bad in (lambda: v.sample(lg.cpu(), u), lambda: v.sample(lg, u.cpu()), lambda: v.sample(lg, u[:1]),
                    lambda: v.sample(lg, u.double()), lambda: v.sample(lg[..., ::2], u),
                    lambda: v.sample(lg.transpose(0, 1), u.T.contiguous()),
                    lambda: v.sample(lg, u, temperature=torch.ones(3, device="cuda")),
                    lambda: v.sample(lg, u, top_k=torch.ones(2, device="cuda")),
                    lambda: v.sample(lg, u, out={"tokens": torch.zeros(2, 3, device="cuda")}),
                    lambda: v.filter_logits(lg, out={"logits": lg.bfloat16()}),
                    lambda: v.filter_logits(lg[0, 0]),
                    lambda: v.logprobs(lg, torch.zeros(2, 3, device="cuda")),
                    lambda: v.logprobs(lg, torch.zeros(2, 3, device="cuda", dtype=torch.int32),
                                       torch.ones(3, device="cuda", dtype=torch.int32))):
            with pytest.raises((ValueError, TypeError)):
                bad()
        with pytest.raises(TypeError):
            v.sample(lg.half(), u)
        with pytest.raises(sv.SpecVerifyError):
            v.sample(lg, u, temperature=-1.0)
