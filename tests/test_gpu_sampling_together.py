"""The sampling calls next to the verify entries they work with, and as programs run them: in a draft
loop, on streams of their own, in graphs, in threads."""
import threading

import numpy as np
import pytest

import oracle
from tests import gpu_helpers as gh
from tests.sampling_reference import MARGIN, row_truth
from tests.test_gpu_sampling import OFF, _f64, _tensor, check_logprobs, check_rows, rows_of, run_all

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _raw(t):
    """As the oracle takes them: bfloat16 by its bits."""
    torch = _torch()
    return t.cpu().view(torch.int16).numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy()


def _numpy(out):
    return {k: t.cpu().numpy() for k, t in out.items()}


def _draft(v, dl, u, settings):
    """K single-row draws at the strides of q [B, K, V] and tokens [B, K]."""
    torch = _torch()
    B, K, V = dl.shape
    q = torch.full((B, K, V), -1.0, device="cuda")
    tok = torch.full((B, K), -1, dtype=torch.int32, device="cuda")
    for i in range(K):
        r = v.sample(dl[:, i], u[:, i], **settings, out={"tokens": tok[:, i], "probs": q[:, i]})
        assert set(r) == {"tokens", "probs"}
    return q, tok


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("settings", [{**OFF, "temperature": 0.7, "top_k": 30},
                                      {**OFF, "temperature": 1.2, "top_p": 0.9, "min_p": 0.01}, OFF],
                         ids=["k", "p", "off"])
def test_a_decode_step(dtype, settings):
    """Draft, truncate the target, verify, and report log-probabilities."""
    torch = _torch()
    B, K, V = 12, 4, 5003
    v = gh.verifier()
    g = torch.Generator(device="cuda").manual_seed(2)
    base = rows_of(B, K + 1, V, 21)
    tl = _tensor(base, dtype)
    dl = _tensor(base[:, :K] + 0.7 * rows_of(B, K, V, 22, 1.0), dtype)
    u = torch.rand(B, 2 * K + 1, device="cuda", generator=g)
    q, tok = _draft(v, dl, u, settings)
    check_rows(dl, settings, u.cpu().numpy(),
               {**_numpy(v.sample(dl, u[:, :K].contiguous(), **settings)), "probs": q.cpu().numpy(), "tokens": tok.cpu().numpy()})
    fil = v.filter_logits(tl, **settings)["logits"]
    uv = u[:, K:].contiguous()
    T = settings["temperature"]
    out = v.run(fil, q, tok, uv, T)
    want = oracle.verify(_raw(fil), dtype, q.cpu().numpy(), tok.cpu().numpy(), uv.cpu().numpy(), T)
    gh.compare(_numpy(out), want, K, check_stats=False)
    assert 1 < int(out["accept_len"].sum()) < B * (K + 1)
    # the drafter's truncated logits stand for the probabilities drawn from
    also = v.run_draft_logits(fil, v.filter_logits(dl, **settings)["logits"], tok, uv, T, T)
    gh.compare(_numpy(also), want, K, check_stats=False)
    for rows in (fil, tl):
        check_logprobs(rows, out["out_tokens"], out["accept_len"], T, 8,
                       v.logprobs(rows, out["out_tokens"], out["accept_len"], temperature=T, top_n=8))
    assert v.error() == (0, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_filtering_and_verifying_is_the_truncated_verify(dtype):
    torch = _torch()
    B, K, V, T, top_p, min_p = 24, 3, 4001, 0.8, 0.9, 0.02
    v = gh.verifier()
    lg = _tensor(rows_of(B, K + 1, V, 5), dtype)
    q = torch.softmax(_tensor(rows_of(B, K, V, 6), "f32"), -1)
    u = torch.rand(B, K + 1, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    tok = torch.multinomial(q.reshape(-1, V), 1, generator=torch.Generator(device="cuda").manual_seed(1))
    tok = tok.reshape(B, K).to(torch.int32)
    want = oracle.verify_truncated(_raw(lg), dtype, q.cpu().numpy(), tok.cpu().numpy(), u.cpu().numpy(), T, top_p,
                                   min_p)
    fil = v.filter_logits(lg, temperature=T, top_p=top_p, min_p=min_p)
    gh.compare(_numpy(v.run(fil["logits"], q, tok, u, T)), want, K, check_stats=False)
    # and by the ragged entry, rows packed
    offsets = (torch.arange(B + 1, device="cuda") * (K + 1)).to(torch.int32)
    out = v.run_ragged(fil["logits"].reshape(-1, V), q.reshape(-1, V), tok.reshape(-1), u.reshape(-1), offsets, K, T)
    out = {"accept_len": out["accept_len"], "out_tokens": out["out_tokens"].reshape(B, K + 1),
           "accept_mask": out["accept_mask"].reshape(B, K), "status": out["status"]}
    gh.compare(_numpy(out), want, K, check_stats=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_temperature_zero_is_the_greedy_verifys_choice(dtype):
    torch = _torch()
    B, K, V = 8, 3, 6007
    x = np.round(rows_of(B, K + 1, V, 3) * 4) / 4  # ties for the largest
    lg = _tensor(x, dtype)
    v = gh.verifier()
    got = v.sample(lg, torch.rand(B, K + 1, device="cuda"), temperature=0.0, probs=True)
    # drafts that the greedy verify accepts one and all: it reaches every row
    out = v.run_greedy(lg, got["tokens"][:, :K].contiguous(), argmax=True)
    assert (out["accept_len"] == K + 1).all() and torch.equal(got["tokens"], out["row_argmax"])
    assert torch.equal(got["tokens"], out["out_tokens"])
    assert torch.equal(got["probs"], torch.nn.functional.one_hot(got["tokens"].long(), V).float())
    assert (got["p_token"] == 1).all() and (got["kept"] == 1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_draws_follow_the_distribution(dtype):
    """N evenly spaced uniforms give a token of probability p within one of N p times; a rounded cut
    point moves one draw more at either end."""
    torch = _torch()
    N, V = 4096, 23
    lg = _tensor(rows_of(1, 1, V, 31, 1.0), dtype)
    u = ((torch.arange(N, device="cuda") + 0.5) / N)[:, None]
    for s in (OFF, {**OFF, "temperature": 0.8, "top_p": 0.85}, {**OFF, "top_k": 5, "min_p": 0.02}):
        t = row_truth(_f64(lg)[0, 0], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
        got = gh.verifier().sample(lg.expand(N, 1, V).contiguous(), u, **s)["tokens"]
        n = np.bincount(got.cpu().numpy()[:, 0], minlength=V)
        assert (np.abs(n - N * t["probs"]) <= 2).all() and (n[~t["keep"]] == 0).all()


@pytest.mark.parametrize("V,cluster,dtype", [(300001, 1, "f32"), (300001, 1, "bf16"), (2000003, 0, "bf16"),
                                             (2000003, 16, "f32"), (300001, 3, "f32"), (1 << 21, 1, "bf16")])
def test_long_rows(V, cluster, dtype):
    """More steps per thread than the first pass keeps codes for, and weights of fewer bits."""
    for s in (OFF, {**OFF, "top_p": 0.9}, {**OFF, "top_k": 50, "top_p": 0.95, "temperature": 0.6}):
        lg = _tensor(rows_of(1, 1, V, V % 7), dtype)
        u, got, fil = run_all(lg, s, cluster=cluster)
        check_rows(lg, s, u, got, fil)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,T", [(3000, 1.0), (20000, 0.7)])
def test_borders(V, T, dtype):
    """top-p and uniforms right beside the steps of the running sum: 2e-7 and 3e-6 of the mass off,
    closer than sums in floats tell."""
    torch = _torch()
    lg = _tensor(rows_of(1, 1, V, 77), dtype)
    l = _f64(lg)[0, 0]
    w = np.sort(np.exp((l - l.max()) / T))[::-1]
    run = np.cumsum(w) / w.sum()
    at = [0, 1, 5, 40, 150, 400, V // 4, V // 2]
    p = np.concatenate([[run[i] - 3e-6, run[i] - 2e-7, run[i] + 2e-7, run[i] + 3e-6] for i in at])
    p = p[(p > 0) & (p < 1)].astype(np.float32)
    B = len(p)
    rows = lg.expand(B, 1, V).contiguous()
    ps = torch.tensor(p, device="cuda")
    s = {**OFF, "temperature": T, "top_p": ps}
    u, got, fil = run_all(rows, s)
    check_rows(rows, s, u, got, fil)
    s = {**OFF, "temperature": T}
    u, got, fil = run_all(rows, s, u=ps[:, None].contiguous())
    check_rows(rows, s, u, got)
    # the same, as draws from a truncated row
    s = {**OFF, "temperature": T, "top_k": V // 2}
    u, got, fil = run_all(rows, s, u=ps[:, None].contiguous())
    check_rows(rows, s, u, got)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_long_tail_of_small_weights(dtype):
    """One token of weight 1 and a tail of equal small ones: float32's sums must not round them away
    one vector at a time.  bfloat16 counts them, and weighs each in whole 2^-43."""
    V, far = 100003, 25.0
    x = np.full((1, 1, V), -far)
    x[0, 0, 1234] = 0.0
    lg = _tensor(x, dtype)
    w = np.exp(-far)
    fil = gh.verifier().filter_logits(lg, top_k=1)
    rel = 1.0 / (1.0 + (V - 1) * w)
    assert abs(float(fil["mass"]) - rel) <= 2.0 ** -24 + 1e-9
    # a uniform in the tail: its entry number is off by the sum's error over an entry's weight at most
    E = 1.0 + (V - 1) * w
    n = 70000
    u = np.float32((1.0 + n * w) / E)
    got = gh.verifier().sample(lg, _tensor([[u]], "f32"))
    j = int(got["tokens"])
    first = (float(u) * E - 1.0) / w
    j = j if j < 1234 else j - 1
    # weights of e^-25 = 2^-36 are good to 2^-44 = 2^-8 of themselves
    assert 0 <= j < V - 1 and abs(j - first) <= 2.0 ** -8 * V + 2


@pytest.mark.parametrize("V,far", [(100003, 25.0), (250000, 25.0)])
def test_a_bfloat16_tail_is_weighed_as_one(V, far):
    """Equal entries in a place of their own: their mass is rounded once, not V times."""
    x = np.full((1, 1, V), 2.0 - far)
    x[0, 0, 1234] = 2.0
    lg = _tensor(x, "bf16")
    w = np.exp(-far)
    E = 1.0 + (V - 1) * w
    for part in (0.2, 0.7, 0.95):
        u = np.float32((1.0 + part * (V - 1) * w) / E)
        j = int(gh.verifier().sample(lg, _tensor([[u]], "f32"))["tokens"])
        j = j if j < 1234 else j - 1
        # the tail to 2^-39 of itself; E and u E to half a unit and a unit of 2^-43
        off = (V - 1) * 2.0 ** -39 + 2 * 2.0 ** -43 / w + 1
        assert abs(j - (float(u) * E - 1.0) / w) <= off


def test_streams_and_threads():
    """Calls on streams of their own, at once, from two threads with one context."""
    torch = _torch()
    v = gh.verifier()
    s = {**OFF, "top_p": 0.9}
    data = []
    for i in range(4):
        lg = _tensor(rows_of(32, 1, 20000 + i, i), "bf16" if i & 1 else "f32")
        data.append((lg, torch.rand(32, 1, device="cuda")))
    torch.cuda.synchronize()
    want = [v.sample(lg, u, **s, probs=True) for lg, u in data]
    wf = [v.filter_logits(lg, **s) for lg, _ in data]
    torch.cuda.synchronize()
    results, errors = {}, []

    def work(j):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for rep in range(5):
                    for i in range(4):
                        lg, u = data[(i + j) % 4]
                        r = v.sample(lg, u, **s, probs=True)
                        f = v.filter_logits(lg, **s)
                        results[j, rep, (i + j) % 4] = (r, f)
            st.synchronize()
        except Exception as e:  # noqa: BLE001 -- shown by the assertion below
            errors.append(e)

    ts = [threading.Thread(target=work, args=(j,)) for j in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors
    for (_, _, i), (r, f) in results.items():
        assert all(torch.equal(r[k], want[i][k]) for k in r) and all(torch.equal(f[k], wf[i][k]) for k in f)


def test_graphs():
    """A decode step's calls captured twice with one context: replays read what the tensors hold
    then, settings included, and give an eager call's bits."""
    torch = _torch()
    v = gh.verifier()
    B, K, V = 6, 2, 9001
    graphs = []
    for n in range(2):
        t = {"tl": _tensor(rows_of(B, K + 1, V, n), "bf16"), "dl": _tensor(rows_of(B, K, V, 9 + n), "bf16"),
             "u": torch.rand(B, 2 * K + 1, device="cuda"), "T": torch.full((B,), 0.8, device="cuda"),
             "k": torch.full((B,), 20, dtype=torch.int32, device="cuda")}

        def step(t=t):
            s = {"temperature": t["T"], "top_k": t["k"], "top_p": 0.95}
            d = v.sample(t["dl"], t["u"][:, :K].contiguous(), **s, probs=True)
            f = v.filter_logits(t["tl"], **s)
            o = v.run(f["logits"], d["probs"], d["tokens"], t["u"][:, K:].contiguous(), 0.8)
            p = v.logprobs(f["logits"], o["out_tokens"], o["accept_len"], temperature=0.8, top_n=4)
            return {**{f"d{k}": x for k, x in d.items()}, **{f"f{k}": x for k, x in f.items()}, **o,
                    **{f"p{k}": x for k, x in p.items()}}

        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            step()
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            out = step()
        graphs.append((g, t, out, step))
    for rep in range(3):
        for n, (g, t, _, _) in enumerate(graphs):
            t["tl"].copy_(_tensor(rows_of(B, K + 1, V, 50 + rep + n), "bf16"))
            t["dl"].copy_(_tensor(rows_of(B, K, V, 60 + rep + n), "bf16"))
            t["u"].uniform_()
            t["k"].fill_(5 + 30 * rep)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for st, (g, _, _, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for _, t, out, step in graphs:
            want = step()
            for k in out:
                assert torch.equal(torch.nan_to_num(out[k].float(), -5.0), torch.nan_to_num(want[k].float(), -5.0)), k


def test_outputs_that_are_left_out():
    torch = _torch()
    v = gh.verifier()
    lg = _tensor(rows_of(3, 2, 4000, 1), "f32")
    u = torch.rand(3, 2, device="cuda")
    s = {**OFF, "top_p": 0.8, "top_k": 100}
    want = v.sample(lg, u, **s, probs=True)
    tok = torch.empty(3, 2, dtype=torch.int32, device="cuda")
    assert set(v.sample(lg, u, **s, out={"tokens": tok})) == {"tokens"} and torch.equal(tok, want["tokens"])
    full = v.filter_logits(lg, **s)
    out = torch.empty_like(lg)
    v.filter_logits(lg, **s, out={"logits": out})
    assert torch.equal(out, full["logits"])
    lp = v.logprobs(lg, tok, top_n=3)
    only = v.logprobs(lg, tok, out={"logprob": torch.empty(3, 2, device="cuda")})
    assert torch.equal(lp["logprob"], only["logprob"])


def test_the_same_row_twice_and_a_row_for_every_sequence():
    """A batch that reads one row many times (stride as for one sequence per row), settings apart."""
    torch = _torch()
    V, B = 7001, 40
    lg = _tensor(rows_of(1, 1, V, 8), "f32").expand(B, 1, V).contiguous()
    ks = torch.arange(1, B + 1, device="cuda", dtype=torch.int32)
    s = {**OFF, "top_k": ks}
    u, got, fil = run_all(lg, s)
    assert (fil["kept"][:, 0] == np.arange(1, B + 1)).all()  # no ties among these
    check_rows(lg, s, u, got, fil)
