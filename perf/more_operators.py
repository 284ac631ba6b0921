"""The losses a drafter is trained with, as a training loop calls them: distillation from the target's
top log-probabilities, and the cross entropy of a vocabulary head that never keeps its logits; each with
its gradients.

Definitions, for a row z of V draft logits at temperature T, q = softmax(z / T), and a teacher's list of
tokens x_k with log-probabilities a_k (entries of token -1 are none), t_k = exp(a_k):
    top:  t_k is divided by the list's sum, L = sum_k t_k (ln t_k - ln q(x_k)), dL/dz_v = (q_v - t_v) / T
    tail: what the list leaves, r = max(0, 1 - sum_k t_k), is one more outcome, of draft mass
          q_rest = sum of q outside the list: L = sum_k t_k (a_k - ln q(x_k)) + r (ln r - ln q_rest),
          dL/dz_v = ((sum_k t_k + r) q_v - t_v) / T on the list and (... q_v - r q_v / q_rest) / T off it
For a row h of a hidden state [R, D], a head's weight W [V, D] and a label y:
    z_v = h . W_v,  L = ln sum_v exp z_v - z_y,  dL/dh = sum_v (p_v - [v = y]) W_v,
    dL/dW_v = sum over rows of (p_v - [v = y]) h
    and beside L the row's lse = ln sum_v exp z_v, which the gradients' call takes.
Rows of no list and of label -1, and those from accept_len on, have loss and lse 0 and no gradient; gradients
are those of sum over rows of (grad_loss times loss).
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
    d = {"op": "distill", "temperature": 1.0, "tail": False, "grad": True, "lens": False}
    c = {"op": "cross_entropy", "lens": False}
    return [
        # one sequence's drafts while a server runs: a drafter that keeps learning, a call's latency
        {"name": "distill 1x5x32000 f32", **d, "B": 1, "K1": 5, "V": 32000, "dtype": "f32", "rows": "normal", "n": 20},
        # a validation step: the loss alone
        {"name": "distill 8x5x32000 bf16 loss", **d, "B": 8, "K1": 5, "V": 32000, "dtype": "bf16", "rows": "peaked", "n": 20,
         "temperature": 0.6, "grad": False},
        # odd sizes, float32, rows that the verify emitted, the tail as one outcome
        {"name": "distill 37x3x50257 f32 tail", **d, "B": 37, "K1": 3, "V": 50257, "dtype": "f32", "rows": "normal", "n": 32,
         "temperature": 0.8, "tail": True, "lens": True},
        # a serving batch's rows, kept as training data
        {"name": "distill 64x4x151936 bf16 tail", **d, "B": 64, "K1": 4, "V": 151936, "dtype": "bf16", "rows": "normal", "n": 20,
         "tail": True},
        # a training step of a large vocabulary
        {"name": "distill 256x8x128256 bf16", **d, "B": 256, "K1": 8, "V": 128256, "dtype": "bf16", "rows": "zipf", "n": 20},
        # the same in float32 with a stored teacher's longer lists
        {"name": "distill 256x8x128256 f32 tail", **d, "B": 256, "K1": 8, "V": 128256, "dtype": "f32", "rows": "zipf", "n": 64,
         "tail": True},
        # one sequence: the loss of a few rows, all of the weight to read
        {"name": "cross entropy 1x5x32000 d1024 loss", **c, "B": 1, "K1": 5, "V": 32000, "D": 1024, "part": "loss"},
        # a small batch learning its head, rows that the verify emitted
        {"name": "cross entropy 8x5x32000 d1024 both", **c, "B": 8, "K1": 5, "V": 32000, "D": 1024, "part": "both", "lens": True},
        # odd sizes everywhere
        {"name": "cross entropy 37x3x50257 d1000 both", **c, "B": 37, "K1": 3, "V": 50257, "D": 1000, "part": "both"},
        # a drafter under the target's own head, which stays as it is
        {"name": "cross entropy 64x4x151936 d2048 hidden", **c, "B": 64, "K1": 4, "V": 151936, "D": 2048, "part": "hidden"},
        # validation of a large batch
        {"name": "cross entropy 256x8x128256 d4096 loss", **c, "B": 256, "K1": 8, "V": 128256, "D": 4096, "part": "loss"},
        # a training step: loss, and the gradients of the hidden states and of the head
        {"name": "cross entropy 1024x8x128256 d4096 both", **c, "B": 1024, "K1": 8, "V": 128256, "D": 4096, "part": "both"},
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    case = {"op": rng.choice(["distill", "cross_entropy"]), "K1": rng.randint(1, 8), "V": _log_int(rng, 1000, 160000),
            "lens": rng.random() < 0.4}
    if case["op"] == "distill":
        case.update(dtype=rng.choice(["bf16", "f32"]), rows=rng.choice(["normal", "peaked", "zipf"]),
                    n=rng.choice([1, 5, 20, 32, 64, 100]), temperature=rng.choice([0.6, 0.8, 1.0, 2.0]),
                    tail=rng.random() < 0.5, grad=rng.random() < 0.75)
        most = 256 * 8 * 128256 // (case["K1"] * case["V"])
        case["B"] = _log_int(rng, 1, min(256, most))
        return case
    case.update(D=8 * _log_int(rng, 8, 512), part=rng.choice(["loss", "hidden", "both"]))
    most = 1024 * 8 * 128256 * 4096 // (case["K1"] * case["V"] * case["D"])
    case["B"] = _log_int(rng, 1, min(1024, most))
    return case


def _logits(case, g, rows):
    """Draft rows as the repository's workloads shape them."""
    x = torch.randn(rows, case["V"], device="cuda", generator=g)
    if case["rows"] == "peaked":  # one entry in a hundred stands out
        return 3.0 * x + 8.0 * (torch.rand(x.shape, device="cuda", generator=g) < 0.01)
    if case["rows"] == "zipf":  # the lower the id, the more frequent the token
        return 2.0 * x - 1.1 * torch.log(torch.arange(1, case["V"] + 1, device="cuda"))
    return 2.5 * x


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * (seed % (1 << 30)) + 29)
    B, K1, V = case["B"], case["K1"], case["V"]
    R = B * K1
    s = {"case": case, "accept_len": None}
    if case["lens"]:
        s["accept_len"] = torch.randint(1, K1 + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
        live = torch.arange(K1, device="cuda")[None] < s["accept_len"][:, None]
    else:
        live = torch.ones(B, K1, device="cuda", dtype=torch.bool)
    # the mean over the rows that count, some of them weighed less
    s["grad_loss"] = ((0.5 + 0.5 * torch.rand(B, K1, device="cuda", generator=g)) / live.sum()).float().contiguous()
    if case["op"] == "distill":
        n, T = case["n"], case["temperature"]
        s["logits"] = torch.empty(R, V, device="cuda", dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        s["top_logprobs"] = torch.empty(R, n, device="cuda")
        s["top_tokens"] = torch.empty(R, n, device="cuda", dtype=torch.int32)
        for a in range(0, R, 256):
            x = _logits(case, g, min(256, R - a))
            s["logits"][a:a + len(x)] = x.to(s["logits"].dtype)
            x += 0.7 * torch.randn(x.shape, device="cuda", generator=g)  # the target, which the drafter resembles
            top = (x / T).log_softmax(-1).topk(n, dim=-1)
            s["top_logprobs"][a:a + len(x)] = top.values
            s["top_tokens"][a:a + len(x)] = top.indices.to(torch.int32)
        for k, w in (("logits", V), ("top_logprobs", n), ("top_tokens", n)):
            s[k] = s[k].view(B, K1, w)
        # logprobs leaves NaN and -1 where the verify emitted nothing
        s["top_logprobs"][~live] = torch.nan
        s["top_tokens"][~live] = -1
        return s
    D = case["D"]
    s["weight"] = (2.0 / D ** 0.5 * torch.randn(V, D, device="cuda", generator=g)).bfloat16()
    labels = torch.randint(0, V, (B, K1), device="cuda", generator=g)
    # a state that leans to its label, some more than others
    lean = 4.0 * torch.rand(R, 1, device="cuda", generator=g)
    h = torch.randn(R, D, device="cuda", generator=g) + lean * s["weight"][labels.view(-1)].float()
    s["hidden"] = h.bfloat16().view(B, K1, D)
    s["labels"] = torch.where(live, labels, -1).to(torch.int32).contiguous()
    return s


def _live(s):
    at = torch.arange(s["case"]["K1"], device="cuda")
    if s["accept_len"] is None:
        return torch.ones(s["case"]["B"], len(at), device="cuda", dtype=torch.bool)
    return at[None] < s["accept_len"][:, None]


def _plain_distill(s):
    case = s["case"]
    B, K1, V, T = case["B"], case["K1"], case["V"], float(np.float32(case["temperature"]))
    x = s["top_tokens"].view(B * K1, -1).long()
    there = x >= 0
    live = _live(s).view(-1, 1) & there.any(-1, keepdim=True)
    there = there & live
    a = torch.where(there, s["top_logprobs"].view(B * K1, -1).double(), -torch.inf)
    t = a.exp()
    if case["tail"]:
        r = (1.0 - t.sum(-1, keepdim=True)).clamp(min=0.0)
    else:
        whole = t.sum(-1, keepdim=True)
        t = torch.where(live, t / whole, 0.0)
        a = torch.where(live, a - whole.log(), -torch.inf)
        r = torch.zeros_like(whole)
    total = t.sum(-1, keepdim=True) + r
    z = s["logits"].view(B * K1, V).float()
    m = z.amax(-1, keepdim=True)
    w = torch.exp((z - m) / T)
    at = torch.where(there, x, 0)
    lw = (z.gather(-1, at) - m).double() / T
    listed = torch.zeros_like(w, dtype=torch.bool).scatter_(-1, torch.where(there, x, x.amax(-1, keepdim=True).clamp(min=0)), True)
    listed &= live
    rest = torch.where(listed, 0.0, w).sum(-1, keepdim=True).double()
    S = rest + torch.where(there, lw.exp(), 0.0).sum(-1, keepdim=True)
    lq = lw - S.log()
    loss = torch.where(t > 0, t * (a - lq), 0.0).sum(-1, keepdim=True)
    loss = loss + torch.where(r > 0, r * (r.log() - (rest / S).log()), 0.0)
    out = {"loss": torch.where(live, loss, 0.0).float().view(B, K1)}
    if case["grad"]:
        g = s["grad_loss"].view(-1, 1).double() / T
        grad = w * (g * (total / S - torch.where(r > 0, r / rest, 0.0))).float()
        on = (g * (total * lq.exp() - t)).float()
        grad.scatter_add_(-1, at, torch.where(there, on - grad.gather(-1, at), 0.0))
        out["grad_logits"] = torch.where(live, grad, 0.0).to(s["logits"].dtype).view(B, K1, V)
    return out


def _plain_cross_entropy(s):
    case = s["case"]
    B, K1, V, D = case["B"], case["K1"], case["V"], case["D"]
    y = s["labels"].view(-1, 1).long()
    live = _live(s).view(-1, 1) & (y >= 0)
    y = y.clamp(min=0)
    h = torch.where(live, s["hidden"].view(-1, D).float(), 0.0)
    W = s["weight"].float()
    z = h @ W.T
    m = z.amax(-1, keepdim=True)
    zy = z.gather(-1, y)
    p = z.sub_(m).exp_()
    S = p.sum(-1, keepdim=True, dtype=torch.float64)
    lse = m.double() + S.log()
    out = {"loss": torch.where(live, lse - zy.double(), 0.0).float().view(B, K1),
           "lse": torch.where(live, lse, 0.0).float().view(B, K1)}
    if case["part"] != "loss":
        p *= (1.0 / S).float()
        p.scatter_add_(-1, y, torch.full_like(zy, -1.0))
        p *= torch.where(live, s["grad_loss"].view(-1, 1), 0.0)
        out["grad_hidden"] = (p @ W).bfloat16().view(B, K1, D)
        if case["part"] == "both":
            out["grad_weight"] = (p.T @ h).bfloat16()
    return out


def run(state):
    case = state["case"]
    if not own:
        return _plain_distill(state) if case["op"] == "distill" else _plain_cross_entropy(state)
    v = _verifier()
    kept = state.setdefault("kept", {})  # a training loop keeps its output buffers and its workspace
    if case["op"] == "distill":
        out = v.distill(state["logits"], state["top_logprobs"], state["top_tokens"], state["accept_len"],
                        temperature=case["temperature"], tail=case["tail"], grad_loss=state["grad_loss"],
                        grad=case["grad"], out=kept.get("out"))
        kept["out"] = out
        return {k: out[k] for k in ("loss", "grad_logits") if k in out}
    B, K1, V, D = case["B"], case["K1"], case["V"], case["D"]
    if "workspace" not in kept:
        kept["workspace"] = v.cross_entropy_workspace(B, K1, V, D, grad=case["part"] != "loss")
    out = v.cross_entropy(state["hidden"], state["weight"], state["labels"], state["accept_len"],
                          workspace=kept["workspace"], out=kept.get("out"))
    kept["out"] = out
    res = {"loss": out["loss"], "lse": out["lse"]}
    if case["part"] != "loss":
        kept["grads"] = v.cross_entropy_grad(state["hidden"], state["weight"], state["labels"], out["lse"],
                                             state["accept_len"], grad_loss=state["grad_loss"],
                                             weight_grad=case["part"] == "both", workspace=kept["workspace"],
                                             out=kept.get("grads"))
        res.update(kept["grads"])
    return res


def work(case):
    rows, V = case["B"] * case["K1"], case["V"]
    # accepted lengths are even over 1..K1: rows from them on are not read
    live = case["B"] * (case["K1"] + 1) / 2 if case["lens"] else rows
    if case["op"] == "distill":
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": live * (V * es + 8 * case["n"]) + rows * (8 + (V * es if case["grad"] else 0)),
                "flops": live * V * (6.0 if case["grad"] else 4.0)}
    D, part = case["D"], case["part"]
    products = {"loss": 1, "hidden": 2, "both": 3}[part]
    out = {"loss": 0, "hidden": rows * D, "both": rows * D + V * D}[part]
    return {"bytes": 2 * (live * D + V * D + out) + 12 * rows, "flops": 2.0 * products * live * V * D}


def exact(case, seed):
    """In 64 bits: distillation row by row on the host, the head's products in blocks of rows."""
    R, K1, V = case["B"] * case["K1"], case["K1"], case["V"]
    if case["op"] == "distill":
        if R * V > 40_000_000:
            return None
        s = prepare(case, seed)
        T = float(np.float32(case["temperature"]))
        z = s["logits"].double().cpu().numpy().reshape(R, V)
        a, x = s["top_logprobs"].double().cpu().numpy().reshape(R, -1), s["top_tokens"].cpu().numpy().reshape(R, -1)
        gl = s["grad_loss"].double().cpu().numpy().reshape(R)
        lens = s["accept_len"].cpu().numpy() if case["lens"] else np.full(case["B"], K1)
        loss, grad = np.zeros(R), np.zeros((R, V)) if case["grad"] else None
        for i in range(R):
            on = x[i] >= 0
            if i % K1 >= lens[i // K1] or not on.any():
                continue
            k, ak = x[i][on], a[i][on]
            zt = z[i] / T
            lq = zt - zt.max()
            lq -= np.log(np.exp(lq).sum())
            q = np.exp(lq)
            off = np.ones(V, bool)
            off[k] = False
            if not case["tail"]:
                ak = ak - np.logaddexp.reduce(ak)
            t = np.exp(ak)
            r = max(0.0, 1.0 - t.sum()) if case["tail"] else 0.0
            loss[i] = (t * (ak - lq[k])).sum()
            d = (t.sum() + r) * q
            d[k] -= t
            if r > 0:
                lrest = np.logaddexp.reduce(lq[off])
                loss[i] += r * (np.log(r) - lrest)
                d[off] -= r * np.exp(lq[off] - lrest)
            if grad is not None:
                grad[i] = gl[i] * d / T
        out = {"loss": loss.reshape(-1, K1)}
        return {**out, "grad_logits": grad.reshape(-1, K1, V)} if case["grad"] else out
    if work(case)["flops"] > 3e12:
        return None
    s = prepare(case, seed)
    W, D = s["weight"].double(), case["D"]
    h, y, gl = s["hidden"].double().view(R, D), s["labels"].long().view(R), s["grad_loss"].double().view(R)
    loss, lse = (torch.zeros(R, device="cuda", dtype=torch.float64) for _ in range(2))
    gh, gw = torch.zeros_like(h), torch.zeros_like(W) if case["part"] == "both" else None
    rows = torch.nonzero(y >= 0)[:, 0]
    for at in rows.split(256):
        lp = h[at] @ W.T
        lse[at] = torch.logsumexp(lp, -1)
        lp -= lse[at, None]
        loss[at] = -lp.gather(-1, y[at, None])[:, 0]
        if case["part"] == "loss":
            continue
        d = lp.exp_()
        d[torch.arange(len(at), device="cuda"), y[at]] -= 1.0
        d *= gl[at, None]
        gh[at] = d @ W
        if gw is not None:
            gw += d.T @ h[at]
    out = {"loss": loss.view(-1, K1), "lse": lse.view(-1, K1)}
    if case["part"] != "loss":
        out["grad_hidden"] = gh.view(-1, K1, D)
        if gw is not None:
            out["grad_weight"] = gw
    return out
