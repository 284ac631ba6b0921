"""The sampling operators as a decode loop calls them: drawing tokens from given uniforms under
temperature, top-k, top-p and min-p (with the drawn-from distribution as draft rows), truncating
logits by the same filters for a verify, and the log-probabilities of the tokens a verify emitted.

Definitions, for a row l of V logits at temperature T > 0:
    w_v = exp((l_v - max l) / T),  S = sum of w
    v is kept when l_v > -inf, fewer than top_k entries are larger than l_v, the mass of the
    entries larger than l_v is below top_p S, and w_v >= min_p (every tie at a border is kept)
    E = sum of w over the kept entries
    sample: the first entry, by descending logit and ascending id, whose running sum of kept
        weights exceeds u E
    filter: l_v where kept, -inf elsewhere
    logprobs: (l_x - max l)/T - ln S, the rank of x, and the n largest entries
"""
import numpy as np
import torch

own = False

_handle = []


def _verifier():
    if not _handle:
        import speculative_decoding_verification_14_gb300 as sv
        _handle.append(sv.Verifier(1 << 12, 32, 1 << 18))
    return _handle[0]


def listed():
    off = {"temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0, "mixed": False}
    return [
        # one sequence drafting its next token at the common server defaults: a call's latency
        {"name": "sample 1x32000 f32", "op": "sample", "B": 1, "K1": 1, "V": 32000, "dtype": "f32", "rows": "normal",
         **off, "top_k": 50, "top_p": 0.95, "probs": False},
        # a small batch of peaked rows, each request with settings of its own (one greedy among them)
        {"name": "sample 8x32000 bf16 mixed", "op": "sample", "B": 8, "K1": 1, "V": 32000, "dtype": "bf16", "rows": "peaked",
         **off, "temperature": 0.6, "mixed": True, "probs": True},
        # a drafter's step for a serving batch at temperature 0.6, top-p 0.95, min-p 0.05, with its q rows
        {"name": "sample 64x151936 bf16 q", "op": "sample", "B": 64, "K1": 1, "V": 151936, "dtype": "bf16", "rows": "normal",
         **off, "temperature": 0.6, "top_p": 0.95, "min_p": 0.05, "probs": True},
        # a large batch of wide rows under top-p alone: tens of thousands of tokens stay in play
        {"name": "sample 256x128256 bf16 top-p", "op": "sample", "B": 256, "K1": 1, "V": 128256, "dtype": "bf16", "rows": "zipf",
         **off, "top_p": 0.95, "probs": False},
        # float32 logits of a vocabulary that is no multiple of anything, no filter: the plain draw
        {"name": "sample 150x50257 f32 open", "op": "sample", "B": 150, "K1": 1, "V": 50257, "dtype": "f32", "rows": "normal",
         **off, "probs": False},
        # the same rows as float32 with every filter on, and q rows
        {"name": "sample 256x128256 f32 all q", "op": "sample", "B": 256, "K1": 1, "V": 128256, "dtype": "f32", "rows": "zipf",
         **off, "top_k": 200, "top_p": 0.9, "min_p": 0.01, "probs": True},
        # one sequence's target rows cut to the top 20 before a verify
        {"name": "filter 1x5x32000 f32", "op": "filter", "B": 1, "K1": 5, "V": 32000, "dtype": "f32", "rows": "normal",
         **off, "top_k": 20},
        # a serving batch's target rows under top-k and top-p
        {"name": "filter 64x4x151936 bf16", "op": "filter", "B": 64, "K1": 4, "V": 151936, "dtype": "bf16", "rows": "normal",
         **off, "temperature": 0.6, "top_k": 50, "top_p": 0.95},
        # the largest batch of target rows under top-p and min-p
        {"name": "filter 256x8x128256 bf16", "op": "filter", "B": 256, "K1": 8, "V": 128256, "dtype": "bf16", "rows": "zipf",
         **off, "top_p": 0.95, "min_p": 0.05},
        # a small batch answering with the five best alternatives of each token
        {"name": "logprobs 8x5x32000 bf16", "op": "logprobs", "B": 8, "K1": 5, "V": 32000, "dtype": "bf16", "rows": "peaked",
         "temperature": 1.0, "top_n": 5},
        # odd sizes, float32
        {"name": "logprobs 37x3x50257 f32", "op": "logprobs", "B": 37, "K1": 3, "V": 50257, "dtype": "f32", "rows": "normal",
         "temperature": 0.8, "top_n": 8},
        # a large batch, twenty alternatives
        {"name": "logprobs 256x8x128256 bf16", "op": "logprobs", "B": 256, "K1": 8, "V": 128256, "dtype": "bf16", "rows": "zipf",
         "temperature": 1.0, "top_n": 20},
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["sample", "sample", "filter", "logprobs"])
    case = {"op": op, "V": _log_int(rng, 1000, 160000), "dtype": rng.choice(["bf16", "f32"]),
            "rows": rng.choice(["normal", "peaked", "zipf"])}
    case["K1"] = 1 if op == "sample" else rng.randint(1, 8)
    most = 256 if op == "sample" else 1500 // case["K1"] if case["dtype"] == "bf16" else 700 // case["K1"]
    case["B"] = _log_int(rng, 1, min(256, most))
    case["temperature"] = rng.choice([0.6, 0.8, 1.0, 1.3])
    if op == "logprobs":
        case["top_n"] = rng.choice([0, 1, 5, 20, 32])
        return case
    case["top_k"] = rng.choice([0, 1, 20, 50, _log_int(rng, 2, 2000)])
    case["top_p"] = rng.choice([1.0, 0.95, 0.9, 0.5])
    case["min_p"] = rng.choice([0.0, 0.05, 0.01])
    if op == "sample":
        case["mixed"] = rng.random() < 0.25
        case["probs"] = rng.random() < 0.5
    else:
        case["mixed"] = False
    return case


def _logits(case, g):
    """Target or draft rows as the repository's workloads shape them."""
    n, V = case["B"] * case["K1"], case["V"]
    out = torch.empty(n, V, device="cuda", dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    for a in range(0, n, 256):
        x = torch.randn(min(256, n - a), V, device="cuda", generator=g)
        if case["rows"] == "peaked":  # one entry in a hundred stands out
            x = 3.0 * x + 8.0 * (torch.rand(x.shape, device="cuda", generator=g) < 0.01)
        elif case["rows"] == "zipf":  # the lower the id, the more frequent the token
            x = 2.0 * x - 1.1 * torch.log(torch.arange(1, V + 1, device="cuda"))
        else:
            x = 2.5 * x
        out[a:a + len(x)] = x.to(out.dtype)
    return out.view(case["B"], case["K1"], V)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * (seed % (1 << 30)) + 17)
    B, K1, V = case["B"], case["K1"], case["V"]
    s = {"case": case, "logits": _logits(case, g)}
    if case["op"] == "logprobs":
        # a verify's answer: the accepted length and the tokens, of plausible ranks; -1 behind the last
        n = torch.randint(1, K1 + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
        top = s["logits"].float().topk(min(V, 40), dim=-1).indices
        pick = torch.randint(0, top.shape[-1], (B, K1, 1), device="cuda", generator=g)
        tokens = top.gather(-1, pick)[..., 0].to(torch.int32)
        s["accept_len"] = n
        s["tokens"] = torch.where(torch.arange(K1, device="cuda")[None] < n[:, None], tokens, -1).to(torch.int32).contiguous()
        return s
    s["args"] = {k: case[k] for k in ("temperature", "top_k", "top_p", "min_p")}
    if case["mixed"]:  # requests of several users in one batch
        i = torch.arange(B, device="cuda")
        s["args"] = {"temperature": (i % 4).float() * 0.3,  # every fourth request is greedy
                     "top_k": torch.tensor([0, 40, 1, 100, 0], device="cuda", dtype=torch.int32)[i % 5].contiguous(),
                     "top_p": torch.tensor([0.95, 1.0, 0.9], device="cuda")[i % 3].contiguous(),
                     "min_p": torch.tensor([0.0, 0.05], device="cuda")[i % 2].contiguous()}
    if case["op"] == "sample":
        s["uniforms"] = torch.rand(B, K1, device="cuda", generator=g)
    return s


def _column(x, B, K1, dtype=torch.float64):
    """A setting for each row, as a column."""
    x = x.to(dtype) if torch.is_tensor(x) else torch.full((B,), x, device="cuda", dtype=dtype)
    return x.repeat_interleave(K1)[:, None]


def _cut(l, args, B, K1):
    """(weights, logits by descending order, their ids, how many are kept, kept mass, whole mass) of rows l [n, V] in 64 bits."""
    n, V = l.shape
    T = _column(torch.tensor(args["temperature"], dtype=torch.float32).double().item() if not torch.is_tensor(args["temperature"])
                else args["temperature"], B, K1)
    k = _column(args["top_k"], B, K1, torch.int64)
    top_p, min_p = _column(args["top_p"], B, K1), _column(args["min_p"], B, K1)
    greedy = T == 0
    z, ids = l.sort(dim=-1, descending=True, stable=True)
    z = z.double()
    w = torch.exp((z - z[:, :1]) / torch.where(greedy, 1.0, T))
    run = w.cumsum(-1)
    whole = run[:, -1:]
    # the first entry of each group of equal logits: what is above the group is above all of it
    at = torch.arange(V, device="cuda")
    first = torch.where(torch.cat([torch.ones_like(z[:, :1], dtype=torch.bool), z[:, 1:] != z[:, :-1]], -1), at, 0).cummax(-1).values
    above = (run - w).gather(-1, first)
    keep = (z > -torch.inf) & ((k <= 0) | (first < k)) & ((top_p >= 1) | (above < top_p * whole)) & (w >= min_p)
    keep = torch.where(greedy, at == 0, keep)
    w = torch.where(greedy, (at == 0).double(), w)
    kept = keep.sum(-1, keepdim=True)
    mass = (w * keep).sum(-1, keepdim=True)
    return w, z, ids, kept, mass, torch.where(greedy, 1.0, whole)


def _plain_sample(s, rows):
    case = s["case"]
    B, K1 = case["B"], case["K1"]
    w, z, ids, kept, mass, _ = _cut(s["logits"].reshape(B * K1, -1), s["args"], B, K1)
    at = torch.arange(w.shape[1], device="cuda")
    w = w * (at < kept)
    u = s["uniforms"].reshape(-1, 1).double()
    i = torch.minimum((w.cumsum(-1) <= u * mass).sum(-1, keepdim=True), kept - 1)
    out = {"tokens": ids.gather(-1, i).to(torch.int32).view(B, K1), "kept": kept.to(torch.int32).view(B, K1),
           "p_token": (w.gather(-1, i) / mass).float().view(B, K1)}
    if rows:
        out["probs"] = torch.zeros_like(w).scatter_(-1, ids, w / mass).float().view(B, K1, -1)
    return out


def _plain_filter(s):
    case = s["case"]
    B, K1 = case["B"], case["K1"]
    l = s["logits"].reshape(B * K1, -1)
    _, _, ids, kept, mass, whole = _cut(l, s["args"], B, K1)
    keep = torch.arange(l.shape[1], device="cuda") < kept
    keep = torch.zeros_like(keep).scatter_(-1, ids, keep)
    return {"logits": torch.where(keep, l, -torch.inf).view(s["logits"].shape), "kept": kept.to(torch.int32).view(B, K1),
            "mass": (mass / whole).float().view(B, K1)}


def _plain_logprobs(s):
    case = s["case"]
    n, V = case["top_n"], case["V"]
    l, x = s["logits"], s["tokens"]
    T = torch.tensor(case["temperature"], dtype=torch.float32).double().item()
    live = torch.arange(case["K1"], device="cuda")[None] < s["accept_len"][:, None]
    d = l.double() - l.amax(-1, keepdim=True).double()
    lp = d / T - torch.exp(d / T).sum(-1, keepdim=True).log()
    at = x.clamp(min=0).long()[..., None]
    lx = l.gather(-1, at)
    out = {"logprob": torch.where(live, lp.gather(-1, at)[..., 0], torch.nan).float(),
           "rank": torch.where(live, 1 + (l > lx).sum(-1), 0).to(torch.int32)}
    if n:
        ids = l.sort(dim=-1, descending=True, stable=True).indices[..., :n]
        out["top_logprobs"] = torch.where(live[..., None], lp.gather(-1, ids), torch.nan).float()
        out["top_tokens"] = torch.where(live[..., None], ids, -1).to(torch.int32)
    return out


def run(state):
    case = state["case"]
    if own:
        v, buffers = _verifier(), state.get("out")  # a decode loop keeps its output buffers
        if case["op"] == "sample":
            out = v.sample(state["logits"], state["uniforms"], **state["args"], probs=case["probs"], out=buffers)
        elif case["op"] == "filter":
            out = v.filter_logits(state["logits"], **state["args"], out=buffers)
        else:
            out = v.logprobs(state["logits"], state["tokens"], state["accept_len"], temperature=case["temperature"],
                             top_n=case["top_n"], out=buffers)
        state["out"] = out
        return {k: x for k, x in out.items() if k != "status"}
    if case["op"] == "sample":
        return _plain_sample(state, case["probs"])
    if case["op"] == "filter":
        return _plain_filter(state)
    return _plain_logprobs(state)


def work(case):
    rows, V, es = case["B"] * case["K1"], case["V"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "sample":
        # a row and its uniform in; token, probability and count out, and the probabilities where they are asked for
        return {"bytes": rows * (V * es + 16 + (4 * V if case["probs"] else 0)), "flops": 4.0 * rows * V}
    if case["op"] == "filter":
        return {"bytes": rows * (2 * V * es + 8), "flops": 4.0 * rows * V}
    # accepted lengths are even over 1..K1: only rows below them are read
    live = case["B"] * (case["K1"] + 1) / 2
    return {"bytes": live * V * es + rows * (12 + 8 * case["top_n"]) + 4 * case["B"], "flops": 4.0 * live * V}


def exact(case, seed):
    """In 64 bits, row by row, with the cut found by its border value instead of by ranks."""
    if case["B"] * case["K1"] * case["V"] > 40_000_000:
        return None
    s = prepare(case, seed)
    l = s["logits"].double().cpu().numpy().reshape(-1, case["V"])
    n, K1 = len(l), case["K1"]

    def setting(name, i):
        x = s["args"][name]
        return float(x[i // K1]) if torch.is_tensor(x) else float(np.float32(x)) if name == "temperature" else float(x)

    if case["op"] == "logprobs":
        T = float(np.float32(case["temperature"]))
        tokens, live = s["tokens"].cpu().numpy().reshape(-1), s["accept_len"].cpu().numpy()
        lp, top = np.full(n, np.nan), np.full((n, case["top_n"]), np.nan)
        for i in range(n):
            if i % K1 < live[i // K1]:
                x = l[i] / T
                lse = x.max() + np.log(np.exp(x - x.max()).sum())
                lp[i] = x[tokens[i]] - lse
                if case["top_n"]:
                    top[i] = np.sort(np.partition(x, -case["top_n"])[-case["top_n"]:])[::-1] - lse
        out = {"logprob": lp.reshape(-1, K1), "rank": None}
        return {**out, "top_logprobs": top.reshape(-1, K1, case["top_n"]), "top_tokens": None} if case["top_n"] else out
    u = s["uniforms"].double().cpu().numpy().reshape(-1) if case["op"] == "sample" else None
    p_token, mass = np.empty(n), np.empty(n)
    full = np.empty_like(l) if case["op"] == "filter" or case["probs"] else None
    for i in range(n):
        x, T, k = l[i], setting("temperature", i), int(setting("top_k", i))
        if T == 0:
            w = np.zeros_like(x)
            w[np.argmax(x)] = 1.0
            keep = w > 0
        else:
            w = np.exp((x - x.max()) / T)
            values, counts = np.unique(x, return_counts=True)  # ascending
            weight = np.exp((values - x.max()) / T) * counts
            above = np.concatenate([np.cumsum(weight[::-1])[::-1][1:], [0.0]])
            more = np.concatenate([np.cumsum(counts[::-1])[::-1][1:], [0]])
            ok = np.exp((values - x.max()) / T) >= setting("min_p", i)
            if k > 0:
                ok &= more < k
            if setting("top_p", i) < 1:
                ok &= above < setting("top_p", i) * weight.sum()
            keep = x >= values[ok].min()
        E = w[keep].sum()
        mass[i] = E / w.sum()
        if u is not None:
            at = np.flatnonzero(keep)
            at = at[np.lexsort((at, -x[at]))]
            run_ = np.cumsum(w[at])
            p_token[i] = w[at[min(np.searchsorted(run_, u[i] * E, side="right"), len(at) - 1)]] / E
        if full is not None:
            full[i] = np.where(keep, x, -np.inf) if u is None else np.where(keep, w / E, 0.0)
    if u is None:
        return {"logits": full.reshape(-1, K1, case["V"]), "kept": None, "mass": mass.reshape(-1, K1)}
    out = {"tokens": None, "kept": None, "p_token": p_token.reshape(-1, K1)}
    return {**out, "probs": full.reshape(-1, K1, case["V"])} if case["probs"] else out
