"""The drafter's losses in 64 bits from their definitions, and how far a float32 kernel may be off.

A weight 2^y with y = (z - m) c: the difference, c and the product round once each (2^-24 of y), the power
is good to 2^-22: off by u_v = 2^-22 + 3 ln2 |y| 2^-24 of itself.  A sum of weights is off by the mean of u_v
over its weights and by the roundings of its additions: a thread adds at most its share of a slice, 54 vectors of
216 KB over 256 threads, and 3 levels of a vector, 5 of a warp, 3 of the warps, 4 of the CTAs, whose joins multiply
by powers that are off by 2^-22 and 3 ln2 |y| 2^-24 again: 69 + 12 (4 + 40) roundings if all of them agree at
|y| below 20; their signs do not, and 128 of 2^-24 are allowed."""
import numpy as np

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
SUM = 128 * 2.0 ** -24


def distill_truth(z, a, x, T=1.0, tail=False, g=1.0):
    """One row: loss, gradient, and bounds on what float32 may be off in either before the last rounding."""
    z, a, x = np.asarray(z, np.float64), np.asarray(a, np.float64), np.asarray(x, np.int64)
    V, T = len(z), float(np.float32(T))
    if (x < -1).any() or (x >= V).any() or len(set(x[x >= 0])) < (x >= 0).sum():
        return {"status": 4}
    on = x >= 0
    x, a = x[on], a[on]
    if not len(x):
        return {"status": 0, "loss": 0.0, "grad": np.zeros(V), "loss_tol": 0.0, "grad_tol": np.zeros(V)}
    if np.isnan(a).any() or (a == np.inf).any() or (not tail and (a == -np.inf).all()) or \
            np.isnan(z).any() or (z == np.inf).any() or (z == -np.inf).all():
        return {"status": 5}
    with np.errstate(all="ignore"):
        t = np.exp(a)
        r = 0.0
        if tail:
            r = max(0.0, 1.0 - t.sum())
        else:
            a = a - a.max()
            a = a - np.log(np.exp(a).sum())
            t = np.exp(a)
        off = np.ones(V, bool)
        off[x] = False
        M = z.max()
        lw = (z - M) / T
        w = np.exp(lw)
        S = w.sum()
        lq = lw - np.log(S)
        q = np.exp(lq)
        mu = z[off].max() if off.any() else -np.inf
        has = mu > -np.inf
        share = np.zeros(V)
        ls = -np.inf
        if has:
            e = np.exp((z[off] - mu) / T)
            share[off] = e / e.sum()
            ls = (mu - M) / T + np.log(e.sum()) - np.log(S)
        if np.exp(ls) < 2.0 ** -126 and r <= 2.0 ** -20:
            r = 0.0
        total = t.sum() + r
        pos = t > 0
        loss = (t[pos] * (a[pos] - lq[x][pos])).sum() + (r * (np.log(r) - ls) if r > 0 else 0.0)
        grad = total * q - r * share
        grad[x] = total * q[x] - t
        # roundings: y in binades against the part's own maximum
        y = np.where(np.isfinite(lw), np.abs(np.where(off, np.where(has, z - mu, 0), z - M)) / T / np.log(2), 0.0)
        u = 2.0 ** -22 + 3 * np.log(2) * y * 2.0 ** -24
        tol_sum = SUM + (q * np.where(np.isfinite(u), u, 0)).sum() + (share * np.where(np.isfinite(u), u, 0)).sum()
        gap = 3 * abs((M - mu) / T) * 2.0 ** -24 if has else 0.0  # the join of the two parts
        tol_sum += min(gap, 2.0 ** -10)
        # shares of the list: expf is good to 2 units in the last place, its argument to |a| 2^-24
        tol_t = t * (2.0 ** -20 + 2 * np.where(pos, np.abs(a), 0) * 2.0 ** -24)
        grad_tol = 4 * tol_sum * (total * q + r * share) + np.where(off, u * np.abs(grad), 0)
        grad_tol[x] = 3 * tol_sum * total * q[x] + q[x] * 2.0 ** -24 * 3 * np.abs(np.where(np.isfinite(lw[x]), lw[x], 0)) + tol_t
        loss_tol = 2 * tol_sum * total
    g = float(np.float32(g))
    return {"status": 0, "loss": loss, "grad": g * grad / T, "loss_tol": loss_tol,
            "grad_tol": abs(g) / T * (grad_tol + 2.0 ** -22 * np.abs(grad))}


def cross_entropy_truth(h, W, y, g=None):
    """Rows h [R, D], weight W [V, D] (64-bit tensors of the stored values), labels y [R] all in [0, V), g [R]:
    everything the two calls give, and bounds before the last rounding of each.

    A logit's products are exact in float32; the tensor cores add them 16 at a time and may cut instead of round:
    (D / 16 + 16) 2^-23 of sum |h| |w|, and the same for the sums of d W and d^T h.  d = g (p - [v = y]):
    p is off by two logits' errors (its own and lse's) and by the power (2^-22 and 3 roundings of |z - lse| log2 e), and d is
    rounded to bfloat16, 2^-8 of itself."""
    import torch
    g = torch.ones(len(h), dtype=torch.float64, device=h.device) if g is None else g.double()
    D, V = h.shape[1], W.shape[0]
    z = h @ W.T
    add = lambda n: (n / 16 + 16) * 2.0 ** -23
    dz = add(D) * (h.abs() @ W.abs().T)
    dz_max = dz.amax(-1)
    lse = torch.logsumexp(z, -1)
    zy = z.gather(-1, y[:, None])[:, 0]
    lse_tol = dz_max + SUM + 2.0 ** -22 + 2.0 ** -24 * lse.abs()
    out = {"lse": lse, "lse_tol": lse_tol, "loss": lse - zy,
           "loss_tol": lse_tol + dz.gather(-1, y[:, None])[:, 0] + 2.0 ** -24 * zy.abs()}
    lp = z - lse[:, None]
    p = lp.exp()
    d = p.clone()
    d[torch.arange(len(h), device=h.device), y] -= 1.0
    rel = torch.expm1(dz + lse_tol[:, None]) + 2.0 ** -22 + 3 * lp.abs() * 2.0 ** -24
    off = p * rel + 2.0 ** -24 * d.abs()
    d, off = d * g[:, None], off * g.abs()[:, None]
    off = off + 2.0 ** -8 * (d.abs() + off) + 2.0 ** -126
    out["grad_hidden"], out["grad_weight"] = d @ W, d.T @ h
    a = d.abs() + off
    # parts of the sums (16 splits, 64 pieces at most) are joined in float32
    out["grad_hidden_tol"] = off @ W.abs() + (add(V) + 80 * 2.0 ** -24) * (a @ W.abs())
    out["grad_weight_tol"] = off.T @ h.abs() + add(len(h)) * (a.T @ h.abs())
    return out
